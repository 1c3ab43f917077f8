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
// p and q converted on their own (to the nearest; exact from 2^-31 on).  So no order
// of summing and no number of CTAs changes a token.
//
// One launch.  A cluster of CTAs shares a request: each finds `a` itself (2 K values),
// sums its part of row a, and gives its sum to the others' shared memory; the part that
// holds the token is read once more, from L2.
//
// Bound by the reads of the two rows: 256 requests of 151936 fp32 entries, 220 MB, in 52 us
// (4.2 TB/s; 32 us at the rate of a plain copy).  A CTA's beginning (starts, drafts and
// their entries, one after another) and end (the cluster's sums, the part read again) read
// little; four CTAs an SM fill some of that.  One request takes 13 us, all of it such
// latency and the launch.
#include <cuda_bf16.h>

#include "vt_device.cuh"
#include "vt_kernels.h"
#include "vt_sampler.h"

namespace vt {
namespace {

constexpr int kVerThreads = 256;
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

// A value v in [0, 2) as a whole number of 2^-54, by three additions whose roundings
// leave multiples of 2^-21, 2^-44 and 2^-54 (of v, of what is left, of what is left of
// that); the rests are exact.  The wholes are the differences of the sums' bits to those
// of the constants, so that sums of wholes are sums of bits.
constexpr float kC1 = 6.f, kC2 = 6.f / (1 << 23), kC3 = 1.5f / (1u << 31);
constexpr uint32_t kB1 = 0x40c00000u, kB2 = 0x35400000u, kB3 = 0x30400000u;  // their bits
__device__ __forceinline__ uint64_t whole(uint32_t s1, uint32_t s2, uint32_t s3) {
  return ((uint64_t)s1 << 33) + (uint64_t)((int64_t)(int32_t)s2 << 10) +
         (uint64_t)(int64_t)(int32_t)s3;
}
__device__ __forceinline__ uint64_t fixed(float v) {
  const float a = __fadd_rn(v, kC1), r = __fsub_rn(v, __fsub_rn(a, kC1));
  const float b = __fadd_rn(r, kC2), q = __fsub_rn(r, __fsub_rn(b, kC2));
  const float c = __fadd_rn(q, kC3);
  return whole(__float_as_uint(a) - kB1, __float_as_uint(b) - kB2, __float_as_uint(c) - kB3);
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t x, uint64_t y) {  // x - y
  uint64_t r;
  const uint64_t minus = 0xbf800000bf800000ull;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(y), "l"(minus), "l"(x));
  return r;
}
// Two values at once into the three sums of bits (out of them for kSign -1).
template <int kSign>
__device__ __forceinline__ void add_bits(uint64_t v, uint32_t (&s)[3]) {
  const uint64_t c1 = 0x40c0000040c00000ull, c2 = 0x3540000035400000ull,
                 c3 = 0x3040000030400000ull;
  const uint64_t a = add2(v, c1), r = sub2(v, sub2(a, c1));
  const uint64_t b = add2(r, c2), q = sub2(r, sub2(b, c2));
  const uint64_t c = add2(q, c3);
  const uint64_t w[3] = {a, b, c};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (kSign > 0) s[i] += (uint32_t)w[i] + (uint32_t)(w[i] >> 32);
    else s[i] -= (uint32_t)w[i] + (uint32_t)(w[i] >> 32);
  }
}

// Values below 2^-8 need two of them: multiples of 2^-31, and the same of 2^-54.  (Nearly
// all entries of a large vocabulary are.  256 requests of 151936 entries: 55 to 52 us.)
constexpr float kLow = 1.f / 256;
template <int kSign>
__device__ __forceinline__ void add_low_bits(uint64_t v, uint32_t (&s)[3]) {
  const uint64_t c1 = 0x3b8000003b800000ull, c3 = 0x3040000030400000ull;  // kLow, kC3
  const uint64_t a = add2(v, c1), r = sub2(v, sub2(a, c1)), c = add2(r, c3);
  if (kSign > 0) {
    s[0] += (uint32_t)a + (uint32_t)(a >> 32);
    s[2] += (uint32_t)c + (uint32_t)(c >> 32);
  } else {
    s[0] -= (uint32_t)a + (uint32_t)(a >> 32);
    s[2] -= (uint32_t)c + (uint32_t)(c >> 32);
  }
}
constexpr uint32_t kBLow = 0x3b800000u;
__device__ __forceinline__ uint64_t whole_low(uint32_t s1, uint32_t s3) {
  return ((uint64_t)s1 << 23) + (uint64_t)(int64_t)(int32_t)s3;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

struct Sum {
  uint64_t mass = 0;
  uint32_t bits = 0;  // of all values, together
  uint32_t over = 0;  // of the masses' upper halves on the way, together
};

// The row that the token is drawn from: p, less q where there is one, without `skip`.
template <typename T>
struct Row {
  const T* p;
  const T* q;
  int skip;
  bool vec;    // 16-byte loads
  bool clamp;  // values below 0 are met: they count as 0
};

// (a NaN stays one)
__device__ __forceinline__ float at_least_0(float v) { return v <= 0.f ? 0.f : v; }

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

// Adds N elements, max(p - q, 0) of each: p less the smaller of p and q.  Values below 0
// and of 2 and more show in `bits` (bits 31 and 30), and the sum is not used then.
template <bool Q, int N>
__device__ __forceinline__ void add_values(const float (&p)[N], const float (&q)[N], Sum& s) {
  uint32_t t[3] = {};
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    s.bits |= __float_as_uint(p[i]) | __float_as_uint(p[i + 1]);
    if constexpr (Q) s.bits |= __float_as_uint(q[i]) | __float_as_uint(q[i + 1]);
    top = max3(top, p[i], p[i + 1]);
  }
  constexpr uint32_t n = Q ? 0 : N;
  if (top < kLow) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      add_low_bits<1>(pair(p[i], p[i + 1]), t);
      if constexpr (Q) add_low_bits<-1>(pair(fminf(p[i], q[i]), fminf(p[i + 1], q[i + 1])), t);
    }
    s.mass += whole_low(t[0] - n * kBLow, t[2] - n * kB3);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      add_bits<1>(pair(p[i], p[i + 1]), t);
      if constexpr (Q) add_bits<-1>(pair(fminf(p[i], q[i]), fminf(p[i + 1], q[i + 1])), t);
    }
    s.mass += whole(t[0] - n * kB1, t[1] - n * kB2, t[2] - n * kB3);
  }
  s.over |= (uint32_t)(s.mass >> 32);
}

__device__ __forceinline__ uint4 load_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Elements [lo, hi) of the row over the lanes of a warp, lo a multiple of 32 E.  A lane
// takes 8 at a time; kStages - 1 of its next loads are under way into 16-byte places of
// its own in shared memory (`ring`: the first, kVerThreads * 16 bytes apart), so that
// nobody waits for another.  (One load ahead in registers, which is what four CTAs an SM
// leave room for: 256 requests of 151936 bf16 entries in 85 us, with the ring 57.)
constexpr int kEach = 8, kStages = 3;  // elements; loads under way and the one in use
template <typename T>
constexpr int ring_bytes() {
  return kStages * 2 * kEach * (int)sizeof(T) * kVerThreads;
}
template <typename T, bool Q>
__device__ __forceinline__ void add_range(const Row<T>& r, int lo, int hi, uint32_t ring, Sum& s) {
  constexpr int E = Wide<T>::E, kStep = 32 * E, kAhead = kEach / E, kNext = kAhead * kStep;
  const int lane = threadIdx.x & 31;
  auto at = [&](int stage, int a, int q) {
    return ring + (uint32_t)((stage * kAhead + a) * 2 + q) * (kVerThreads * 16);
  };
  auto load = [&](int stage, int j0) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int j = j0 + a * kStep + lane * E;
      if (r.vec && j + E <= hi) {
        copy16(at(stage, a, 0), r.p + j);
        if constexpr (Q) copy16(at(stage, a, 1), r.q + j);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i, lo + i * kNext);
  int stage = 0;
#pragma unroll 1
  for (int j0 = lo; j0 < hi; j0 += kNext) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    float x[kEach], y[kEach];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int j = j0 + a * kStep + lane * E;
      float p[E], q[E];
      if (r.vec && j + E <= hi) {
        Wide<T>::split(load_shared(at(stage, a, 0)), p);
        if constexpr (Q) Wide<T>::split(load_shared(at(stage, a, 1)), q);
      } else {
        load_part(r.p, j, hi, false, p);
        if constexpr (Q) load_part(r.q, j, hi, false, q);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        x[a * E + i] = p[i];
        y[a * E + i] = Q ? q[i] : 0.f;
      }
    }
    if (r.clamp)
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        x[i] = at_least_0(x[i]);
        if constexpr (Q) y[i] = at_least_0(y[i]);
      }
    load(stage == 0 ? kStages - 1 : stage - 1, j0 + (kStages - 1) * kNext);
    stage = stage == kStages - 1 ? 0 : stage + 1;
    add_values<Q, kEach>(x, y, s);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!Q && r.skip >= lo && r.skip < hi && lane == (r.skip - lo) / E % 32)
    s.mass -= fixed(r.clamp ? at_least_0(Wide<T>::one(r.p[r.skip])) : Wide<T>::one(r.p[r.skip]));
}
template <typename T>
__device__ __forceinline__ void add_range(const Row<T>& r, int lo, int hi, uint32_t ring, Sum& s) {
  if (r.q) add_range<T, true>(r, lo, hi, ring, s);
  else add_range<T, false>(r, lo, hi, ring, s);
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
__global__ void __launch_bounds__(kVerThreads, 4) verify_kernel(VerifyArgs a) {
  constexpr int E = Wide<T>::E, kStep = 32 * E;
  __shared__ int s_accepted;
  __shared__ uint64_t s_warp[kVerWarps];
  // of each CTA of the cluster: its sum, and what was met; by turns
  __shared__ uint64_t s_mass[2][kVerMaxCtas], s_bad[2][kVerMaxCtas];
  __shared__ uint32_t s_bits[kVerWarps];
  __shared__ float s_rough[kVerWarps];
  extern __shared__ __align__(16) unsigned char s_ring[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = smem_addr(s_ring) + tid * 16;
  const int ctas = a.ctas, rank = (int)cluster_ctarank();
  const int b = blockIdx.x / ctas;
  const int K = a.K;
  cluster_arrive();  // (the others' shared memory may be written behind the wait)

  // ---- how many drafts are accepted
  // (what does not depend on anything is asked for at once)
  const int32_t* tokens = a.tokens + (int64_t)b * K;
  const float* uniforms = a.uniforms + (int64_t)b * (K + 1);
  int x = -1;
  float u = 0.f;
  if (warp == 0 && lane < K) {
    x = tokens[lane];
    u = uniforms[lane];
  }
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
  if (draft) draft += b * a.d_batch;
  if (warp == 0) {
    int first = rows ? n : 0;
    for (int i0 = 0; i0 < first; i0 += 32) {
      const int i = i0 + lane;
      bool no = false;
      if (i0 > 0 && i < n) {
        x = tokens[i];
        u = uniforms[i];
      }
      if (i < n) {
        no = true;
        if (x >= 0 && x < a.V) {
          const double p = Wide<T>::one(target[i * a.t_row + x]);
          const double q = draft ? Wide<T>::one(draft[i * a.d_row + x]) : 1.f;
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
  row.clamp = false;
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
  for (int round = 0;; ++round) {  // (four at most)
    Sum s;
    int lo, hi;
    warp_range(warp, lo, hi);
    if (rows) add_range(row, lo, hi, ring, s);
    // the sum, roughly, where a lane's may not have fit: large
    const float rough =
        warp_sum_f(s.over & 0xc0000000u ? 1e9f : (float)(uint32_t)(s.mass >> 44) * (1.f / 1024.f));
    const uint64_t mass = warp_sum_u64(s.mass);
    const uint32_t bits = __reduce_or_sync(0xffffffffu, s.bits);
    __syncthreads();
    if (lane == 0) {
      s_warp[warp] = mass;
      s_bits[warp] = bits;
      s_rough[warp] = rough;
    }
    __syncthreads();
    const int turn = round & 1;
    if (warp == 0) {
      const uint64_t m = warp_sum_u64(lane < kVerWarps ? s_warp[lane] : 0);
      const uint32_t any = __reduce_or_sync(0xffffffffu, lane < kVerWarps ? s_bits[lane] : 0u);
      const float r = warp_sum_f(lane < kVerWarps ? s_rough[lane] : 0.f);
      // the sum in whole units (bits 0..19), values below 0 (20..), no probabilities (32..)
      const uint64_t flag = (uint64_t)fminf(r, 1024.f) + ((uint64_t)(any >> 31) << 20) +
                            ((uint64_t)((any >> 30) & 1) << 32);
      if (lane < ctas) {
        store_remote(&s_mass[turn][rank], lane, m);
        store_remote(&s_bad[turn][rank], lane, flag);
      }
    }
    cluster_arrive();
    cluster_wait();
    total = before = 0;
    uint64_t flags = 0;
    for (int c = 0; c < ctas; ++c) {
      const uint64_t m = s_mass[turn][c];
      if (c < rank) before += m;
      if (c == rank) mine = m;
      total += m;
      flags += s_bad[turn][c];
    }
    if (((flags >> 20) & 0xfff) != 0 && !row.clamp) {
      row.clamp = true;
      continue;
    }
    bad = (flags >> 32) != 0 || (flags & 0xfffff) >= 512;
    // nothing left of the target's row (a drafter above it everywhere): drawn from it
    // as it is
    if (bad || total != 0 || !(row.q || row.skip >= 0)) break;
    row.q = nullptr;
    row.skip = -1;
    row.clamp = false;
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

  // ---- the token: the warp's chunk, a part of it, the block, the lane, the element
  uint64_t left = t - before;
  int w = 0;
  while (w + 1 < kVerWarps && left >= s_warp[w]) left -= s_warp[w++];
  int lo, hi;
  warp_range(w, lo, hi);
  const int part = (chunk / kStep + kVerWarps - 1) / kVerWarps * kStep;
  __syncthreads();  // (s_warp is written again)
  const int p_lo = min(lo + warp * part, hi), p_hi = min(p_lo + part, hi);
  Sum s;
  add_range(row, p_lo, p_hi, ring, s);
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
    uint64_t each[E], own = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (row.clamp) p[i] = at_least_0(p[i]);
      each[i] = j + i == row.skip ? 0 : fixed(p[i]);
      if (row.q) each[i] -= fixed(fminf(p[i], row.clamp ? at_least_0(q[i]) : q[i]));
      own += each[i];
    }
    const uint64_t upto = warp_scan_u64(own);
    const uint64_t block = __shfl_sync(0xffffffffu, upto, 31);
    if (left >= block) {
      left -= block;
      continue;
    }
    if (left < upto && left >= upto - own) {
      uint64_t rest = left - (upto - own);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (rest < each[i]) {
          out[acc] = j + i;
          break;
        }
        rest -= each[i];
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
  cfg.dynamicSmemBytes = ring_bytes<T>();
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

template <typename T>
cudaError_t prepare_typed() {
  const cudaError_t e = cudaFuncSetAttribute(
      verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(verify_kernel<T>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     ring_bytes<T>());
}

}  // namespace

cudaError_t prepare_verify() {
  const cudaError_t e = prepare_typed<float>();
  return e != cudaSuccess ? e : prepare_typed<__nv_bfloat16>();
}

cudaError_t launch_verify(VerifyArgs a, int dtype, int num_sms, cudaStream_t stream) {
  // CTAs to a request until there are four for every SM, 4096 elements to each at least;
  // more than that, so that some begin when others end, only where each still has 128 KB
  // of a row: 64 requests of 151936 bf16 entries take 24 us with 8 CTAs each and 32 with
  // 16 (19 KB), 512 fp32 ones 134 us with 2 (300 KB) and 157 with 1.
  a.ctas = 1;
  const int64_t row = (int64_t)a.V * (dtype == VT_DTYPE_F32 ? 4 : 2), room = 4ll * num_sms;
  while (a.ctas < kVerMaxCtas && a.ctas * (int64_t)a.B < room && a.V / a.ctas >= 8192 &&
         (2ll * a.ctas * a.B <= room || row / (2 * a.ctas) >= 128 << 10))
    a.ctas *= 2;
  return dtype == VT_DTYPE_F32 ? launch_typed<float>(a, stream)
                               : launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace vt
