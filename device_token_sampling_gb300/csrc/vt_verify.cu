// vt_verify.cu -- drafted tokens against the target's probabilities, from given
// uniform numbers.
//
// Request b has n drafts x_0 .. x_{n-1}, the target's rows p_0 .. p_n and the
// drafter's rows q_0 .. q_{n-1} (a lookup without probabilities: all of q_i on x_i).
// Draft i is accepted when u_i q_i(x_i) < p_i(x_i); the first that is not, a, ends the
// drafts, and the token behind the accepted ones is drawn from r = max(p_a - q_a, 0),
// or from r = p_n when all were accepted:
//   token = the first j with r_0 + .. + r_j > u * (r_0 + .. + r_{V-1}).
// The tokens then have the target's distribution.  Both decisions are exact: the
// product of two 24-bit mantissas fits 64 bits, and the sums are integers of 2^-54,
// p and q converted on their own (values below 2^-31 are cut to 2^-54).  So no order
// of summing and no number of CTAs changes a token.
//
// One launch.  A cluster of CTAs shares a request: each finds `a` itself (2 K values),
// sums its part of row a, and gives its sum to the others' shared memory; the part that
// holds the token is read once more, from L2.
#include <cuda_bf16.h>

#include "vt_device.cuh"
#include "vt_kernels.h"
#include "vt_sampler.h"

namespace vt {
namespace {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerMaxCtas = 16;

template <typename T>
struct Wide;  // 16 bytes of a row
template <>
struct Wide<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void split(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float one(float v) { return v; }
};
template <>
struct Wide<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void split(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
};

// (these shifts give 0 for amounts of 32 and more)
__device__ __forceinline__ uint32_t shl_clamped(uint32_t x, uint32_t n) {
  uint32_t r;
  asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(n));
  return r;
}
__device__ __forceinline__ uint32_t shr_clamped(uint32_t x, uint32_t n) {
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(n));
  return r;
}
// v in units of 2^-54, 0 <= v < 2: mantissa * 2^(exponent - 96), of which one of the
// two terms is 0.
__device__ __forceinline__ void add_fixed(float v, uint64_t& sum, uint32_t& small) {
  const uint32_t b = __float_as_uint(v), e = b >> 23, m = (b & 0x7fffffu) | 0x800000u;
  sum += (uint64_t)m * shl_clamped(1u, e - 96u);
  small += shr_clamped(m >> 1, 95u - e);
}

struct Sum {
  uint64_t mass = 0;
  uint32_t top = 0;   // the largest magnitude's bits
  float rough = 0.f;  // tells a sum that would not fit
};

// The row that the token is drawn from: p, less q where there is one, without `skip`.
template <typename T>
struct Row {
  const T* p;
  const T* q;
  int skip;
  bool vec;  // 16-byte loads
};

// Adds the elements of a lane's E of a block of 32 E (from element j, below `end`).
template <typename T, bool Q>
__device__ __forceinline__ void add_block(const float (&p)[Wide<T>::E], const float (&q)[Wide<T>::E],
                                          int j, int skip, Sum& s) {
  constexpr int E = Wide<T>::E;
  uint64_t less = 0;
  uint32_t small = 0, small_less = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    s.top = max(s.top, __float_as_uint(p[i]) & 0x7fffffffu);
    if constexpr (Q) {
      s.top = max(s.top, __float_as_uint(q[i]) & 0x7fffffffu);
      const float b = fmaxf(q[i], 0.f);
      const bool more = p[i] > b;
      const float v = more ? p[i] : 0.f;
      add_fixed(v, s.mass, small);
      add_fixed(more ? b : 0.f, less, small_less);
      s.rough += v;
    } else {
      const float v = j + i == skip ? 0.f : fmaxf(p[i], 0.f);
      add_fixed(v, s.mass, small);
      s.rough += v;
    }
  }
  s.mass += small;
  if constexpr (Q) s.mass -= less + small_less;
}

// A lane's E elements from j on, zeros past `end`.
template <typename T>
__device__ __forceinline__ void load_part(const T* row, int j, int end, bool vec,
                                          float (&x)[Wide<T>::E]) {
  constexpr int E = Wide<T>::E;
  if (vec && j + E <= end) {
    Wide<T>::split(__ldg(reinterpret_cast<const uint4*>(row + j)), x);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = j + i < end ? Wide<T>::one(row[j + i]) : 0.f;
  }
}

// Elements [lo, hi) of the row over the lanes of a warp; lo a multiple of 32 E.
template <typename T, bool Q>
__device__ __forceinline__ void add_range(const Row<T>& r, int lo, int hi, Sum& s) {
  constexpr int E = Wide<T>::E, kStep = 32 * E, kAhead = Q ? 2 : 4;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int j0 = lo; j0 < hi; j0 += kAhead * kStep) {
    float p[kAhead][E], q[kAhead][E];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int j = j0 + a * kStep + lane * E;
      load_part(r.p, j, hi, r.vec, p[a]);
      if constexpr (Q) load_part(r.q, j, hi, r.vec, q[a]);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      add_block<T, Q>(p[a], q[a], j0 + a * kStep + lane * E, r.skip, s);
  }
}
template <typename T>
__device__ __forceinline__ void add_range(const Row<T>& r, int lo, int hi, Sum& s) {
  if (r.q) add_range<T, true>(r, lo, hi, s);
  else add_range<T, false>(r, lo, hi, s);
}

__device__ __forceinline__ uint64_t warp_scan_u64(uint64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// floor(u * total), total >= 1; u below 0 and NaN count as 0, 1 and more as what draws
// the last element.
__device__ __forceinline__ uint64_t target_of(float u, uint64_t total) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return total - 1;
  const uint32_t b = __float_as_uint(u), e = b >> 23;
  if (e == 0) return 0;  // (below 2^-126)
  const uint64_t m = (b & 0x7fffffu) | 0x800000u;
  const uint64_t hi = __umul64hi(total, m), lo = total * m;
  const uint32_t s = 150 - e;  // at least 24
  if (s < 64) return (hi << (64 - s)) | (lo >> s);
  return s < 128 ? hi >> (s - 64) : 0;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 8 bytes into the same place of another CTA's shared memory.
__device__ __forceinline__ void store_remote(uint64_t* at, uint32_t rank, uint64_t v) {
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, %1;\n\t"
      "st.shared::cluster.u64 [r], %2;\n\t}" ::"r"(smem_addr(at)),
      "r"(rank), "l"(v)
      : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(VerifyArgs a) {
  constexpr int E = Wide<T>::E, kStep = 32 * E;
  __shared__ int s_accepted;
  __shared__ uint64_t s_warp[kVerWarps];
  // of each CTA of the cluster: its sum, and 1 where a value is not a probability; two
  // rounds, the second where the difference has no mass
  __shared__ uint64_t s_mass[2][kVerMaxCtas], s_bad[2][kVerMaxCtas];
  __shared__ uint32_t s_wrong[kVerWarps];
  __shared__ float s_rough[kVerWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = a.ctas, rank = (int)cluster_ctarank();
  const int b = blockIdx.x / ctas;
  const int K = a.K;
  cluster_arrive();  // (the others' shared memory may be written behind the wait)

  // ---- how many drafts are accepted
  int n = a.lens ? min(max(a.lens[b], 0), K) : K;
  const T* target;
  bool rows = true;
  if (a.starts) {
    const int64_t r0 = a.starts[b], r1 = a.starts[b + 1];
    rows = r0 >= 0 && r0 < r1 && r1 <= a.rows;
    n = (int)min((int64_t)n, max(r1 - r0 - 1, (int64_t)0));
    target = static_cast<const T*>(a.target) + r0 * a.t_row;
  } else {
    target = static_cast<const T*>(a.target) + b * a.t_batch;
  }
  const T* draft = static_cast<const T*>(a.draft);
  const int32_t* tokens = a.tokens + (int64_t)b * K;
  const float* uniforms = a.uniforms + (int64_t)b * (K + 1);
  if (draft) draft += b * a.d_batch;
  if (warp == 0) {
    int first = rows ? n : 0;
    for (int i0 = 0; i0 < first; i0 += 32) {
      const int i = i0 + lane;
      bool no = false;
      if (i < n) {
        const int x = tokens[i];
        no = true;
        if (x >= 0 && x < a.V) {
          const double p = Wide<T>::one(target[i * a.t_row + x]);
          const double q = draft ? Wide<T>::one(draft[i * a.d_row + x]) : 1.f;
          const float u = uniforms[i];
          no = !((u > 0.f ? (double)u : 0.) * q < p);
        }
      }
      const unsigned some = __ballot_sync(0xffffffffu, no);
      if (some) first = i0 + __ffs(some) - 1;
    }
    if (lane == 0) s_accepted = first;
  }
  __syncthreads();
  const int acc = s_accepted;

  // ---- the sums of this CTA's part of the row
  const bool refused = acc < n;
  Row<T> row;
  row.p = target + acc * a.t_row;
  row.q = refused && draft ? draft + acc * a.d_row : nullptr;
  row.skip = refused && !draft ? tokens[acc] : -1;
  row.vec = a.vec;
  // whole blocks to a warp
  const int chunk = ((a.V + ctas * kVerWarps - 1) / (ctas * kVerWarps) + kStep - 1) / kStep * kStep;
  const int64_t from = (int64_t)rank * kVerWarps * chunk;
  auto warp_range = [&](int w, int& lo, int& hi) {
    lo = (int)min(from + (int64_t)w * chunk, (int64_t)a.V);
    hi = (int)min((int64_t)lo + chunk, (int64_t)a.V);
  };
  uint64_t total = 0, before = 0, mine = 0;
  bool bad = false;
  cluster_wait();
  for (int round = 0; round < 2; ++round) {
    Sum s;
    int lo, hi;
    warp_range(warp, lo, hi);
    if (rows) add_range(row, lo, hi, s);
    const uint64_t mass = warp_sum_u64(s.mass);
    const float rough = warp_sum_f(s.rough);
    const uint32_t top = __reduce_max_sync(0xffffffffu, s.top);
    __syncthreads();
    if (lane == 0) {
      s_warp[warp] = mass;
      // 2 and more, infinities and NaN; or a sum that may not fit
      s_wrong[warp] = top >= 0x40000000u || !(rough < 512.f);
      s_rough[warp] = rough;
    }
    __syncthreads();
    if (warp == 0) {
      const uint64_t m = warp_sum_u64(lane < kVerWarps ? s_warp[lane] : 0);
      const uint32_t wrong = __any_sync(0xffffffffu, lane < kVerWarps && s_wrong[lane]);
      const float r = warp_sum_f(lane < kVerWarps ? s_rough[lane] : 0.f);
      // (the rough sum travels beside the flag, in whole units)
      const uint64_t flag = wrong || !(r < 512.f) ? 1u << 20 : (uint32_t)r;
      if (lane < ctas) {
        store_remote(&s_mass[round][rank], lane, m);
        store_remote(&s_bad[round][rank], lane, flag);
      }
    }
    cluster_arrive();
    cluster_wait();
    total = before = 0;
    uint64_t flags = 0;
    for (int c = 0; c < ctas; ++c) {
      const uint64_t m = s_mass[round][c];
      if (c < rank) before += m;
      if (c == rank) mine = m;
      total += m;
      flags += s_bad[round][c];
    }
    bad = flags >= 512;
    // nothing left of the target's row (a drafter above it everywhere): drawn from it
    // as it is
    if (bad || total != 0 || !refused) break;
    row.q = nullptr;
    row.skip = -1;
  }

  // ---- the outputs
  const bool none = !rows || bad || total == 0;
  int32_t* out = a.out_tokens + (int64_t)b * (K + 1);
  if (rank == 0) {
    for (int i = tid; i <= K; i += kVerThreads)
      if (i != acc || none) out[i] = i < acc ? tokens[i] : -1;
    if (tid == 0) {
      a.out_accepted[b] = acc;
      a.row_status[b] = bad ? kRowNonfinite : none ? kRowEmpty : kRowOk;
    }
  }
  if (none) return;
  const uint64_t t = target_of(uniforms[K], total);
  if (t < before || t - before >= mine) return;

  // ---- the token: the warp's chunk, a sixteenth of it, the block, the lane, the element
  uint64_t left = t - before;
  int w = 0;
  while (w + 1 < kVerWarps && left >= s_warp[w]) left -= s_warp[w++];
  int lo, hi;
  warp_range(w, lo, hi);
  const int part = (chunk / kStep + kVerWarps - 1) / kVerWarps * kStep;
  __syncthreads();  // (s_warp is written again)
  const int p_lo = min(lo + warp * part, hi), p_hi = min(p_lo + part, hi);
  Sum s;
  add_range(row, p_lo, p_hi, s);
  const uint64_t mass = warp_sum_u64(s.mass);
  if (lane == 0) s_warp[warp] = mass;
  __syncthreads();
  for (int v = 0; v < warp; ++v) {
    if (left < s_warp[v]) return;
    left -= s_warp[v];
  }
  if (left >= s_warp[warp]) return;
#pragma unroll 1
  for (int j0 = p_lo; j0 < p_hi; j0 += kStep) {
    const int j = j0 + lane * E;
    float p[E], q[E];
    load_part(row.p, j, p_hi, row.vec, p);
    if (row.q) load_part(row.q, j, p_hi, row.vec, q);
    Sum own;
    if (row.q) add_block<T, true>(p, q, j, row.skip, own);
    else add_block<T, false>(p, q, j, row.skip, own);
    const uint64_t upto = warp_scan_u64(own.mass);
    const uint64_t block = __shfl_sync(0xffffffffu, upto, 31);
    if (left >= block) {
      left -= block;
      continue;
    }
    if (left < upto && left >= upto - own.mass) {
      uint64_t rest = left - (upto - own.mass);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        // the element alone, by the same arithmetic
        float pe[E] = {}, qe[E] = {};
        pe[0] = p[i];
        if (row.q) qe[0] = q[i];
        Sum e;
        if (row.q) add_block<T, true>(pe, qe, j + i, row.skip, e);
        else add_block<T, false>(pe, qe, j + i, row.skip, e);
        if (rest < e.mass) {
          out[acc] = j + i;
          break;
        }
        rest -= e.mass;
      }
    }
    break;
  }
}

template <typename T>
cudaError_t launch_typed(const VerifyArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)(a.B * a.ctas));
  cfg.blockDim = dim3(kVerThreads);
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t prepare_verify() {
  const auto attr = cudaFuncAttributeNonPortableClusterSizeAllowed;
  const cudaError_t e = cudaFuncSetAttribute(verify_kernel<float>, attr, 1);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(verify_kernel<__nv_bfloat16>, attr, 1);
}

cudaError_t launch_verify(VerifyArgs a, int dtype, int num_sms, cudaStream_t stream) {
  // CTAs to a request until there are two for every SM, 4096 elements to each at least
  a.ctas = 1;
  while (a.ctas < kVerMaxCtas && (int64_t)a.ctas * a.B < 2 * num_sms && a.V / a.ctas >= 8192)
    a.ctas *= 2;
  return dtype == VT_DTYPE_F32 ? launch_typed<float>(a, stream)
                               : launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace vt
