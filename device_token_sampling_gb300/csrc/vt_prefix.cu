// vt_prefix.cu -- single-token attention over a paged cache whose first
// prefix_len tokens are the same for every request.
//
// For request b, head h: out = sum_j p_j v_j / sum_j p_j over positions
// j < len_b, p_j = exp(scale q . k_j - max).  A part of the positions gives
// (max, sum p, sum p v); parts are joined by rescaling to the common maximum.
// The prefix is one part list for all requests (its rows are the B * G query
// heads of a kv head), the rest of each request another.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "vt_device.cuh"
#include "vt_paged.h"
#include "vt_sampler.h"

namespace vt {
namespace {

constexpr int kRows = 16;      // query rows of a unit (one mma tile)
constexpr int kGroup = 16;     // tokens a warp takes at a time
constexpr int kSplitWarps = 4;
constexpr int kStages = 3;

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t* a, uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t* a, uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

template <int D>
struct SplitSmem {
  static constexpr int kPitch = D + 8;                      // elements: rows 16 bytes apart in banks
  static constexpr int kTile = kGroup * kPitch;             // elements of K (or V) of a group
  static constexpr int kWarpElems = kStages * 2 * kTile;
  static constexpr int kQElems = kRows * kPitch;
  static constexpr size_t kBytes = 2 * ((size_t)kSplitWarps * kWarpElems + kQElems);
  static_assert(kWarpElems * 2 >= kRows * D * 4, "a warp's stages hold its accumulators");
};

// One unit: 16 query rows of one kv head against the tokens [t0, t1) of one
// table.  Each of the four warps takes every fourth group of 16 tokens through
// its own ring of bulk copies, with its own running maximum and sum; the four
// are joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(kSplitWarps * 32) split_kernel(AttnArgs a) {
  using S = SplitSmem<D>;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ uint64_t bars[kSplitWarps][kStages];
  __shared__ float s_m[kSplitWarps][kRows], s_l[kSplitWarps][kRows];
  __shared__ int s_lim[kRows];
  __shared__ uint32_t s_mask[kSplitWarps][kStages];
  T* sq = reinterpret_cast<T*>(dyn);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  T* ring = sq + S::kQElems + warp * S::kWarpElems;

  // which unit
  int u = blockIdx.x;
  const int n_prefix_units = a.prefix_mma ? 0 : a.prefix_tiles * a.hkv * a.prefix_splits;
  const bool prefix = u < n_prefix_units;
  int kvh, tile, split, b0 = 0, t0, t1;
  const int32_t* table;
  if (prefix) {
    kvh = u % a.hkv;
    tile = (u / a.hkv) % a.prefix_tiles;
    split = u / (a.hkv * a.prefix_tiles);
    table = a.prefix_blocks;
    t0 = split * a.prefix_chunk;
    t1 = min(t0 + a.prefix_chunk, a.prefix_len);
  } else {
    u -= n_prefix_units;
    kvh = u % a.hkv;
    tile = (u / a.hkv) % a.own_tiles;
    b0 = (u / (a.hkv * a.own_tiles)) % a.B;
    split = u / (a.hkv * a.own_tiles * a.B);
    table = a.table + (int64_t)b0 * a.ld_table;
    const int len = min(max(a.seq_lens[b0], 0), a.cols << a.shift);
    const int base = a.prefix_len & ~(kGroup - 1);
    // a longer request than the host reckoned with gets longer splits
    const int even = ((len - base + a.own_splits - 1) / a.own_splits + kGroup - 1) &
                     ~(kGroup - 1);
    const int chunk = max(a.own_chunk, even);
    const int64_t lo = base + (int64_t)split * chunk;
    t0 = (int)(lo < a.prefix_len ? a.prefix_len : lo < len ? lo : len);
    t1 = (int)(lo + chunk < len ? lo + chunk : len);
  }
  const int n_rows = prefix ? a.B * a.G : a.G;
  if (tid < kRows) {
    const int r = tile * kRows + tid;
    int lim = 0;
    if (r < n_rows) lim = prefix ? min(max(a.seq_lens[r / a.G], 0), a.prefix_len) : t1;
    s_lim[tid] = lim;
  }
  for (int i = tid; i < kRows * (D / 8); i += kSplitWarps * 32) {
    const int r = tile * kRows + i / (D / 8), c = (i % (D / 8)) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < n_rows) {
      const int b = prefix ? r / a.G : b0, g = prefix ? r % a.G : r;
      v = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + b * a.q_row +
                                          (kvh * a.G + g) * a.q_head + c);
    }
    *reinterpret_cast<uint4*>(sq + (i / (D / 8)) * S::kPitch + c) = v;
  }
  if (lane < kStages) mbar_init(&bars[warp][lane], 1);
  fence_mbar_init();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  int hi_lim = 0, lo_lim = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    hi_lim = max(hi_lim, s_lim[i]);
    if (tile * kRows + i < n_rows) lo_lim = min(lo_lim, s_lim[i]);
  }
  t1 = min(t1, hi_lim);

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int row0 = lane >> 2;
  const int lim[2] = {s_lim[row0], s_lim[row0 + 8]};

  if (t0 < t1) {
    uint32_t qf[D / 16][4];
    {
      const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = (lane >> 4) * 8;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        ldsm_x4(qf[ks], smem_addr(sq + r * S::kPitch + ks * 16 + c));
    }
    const int g_first = (t0 >> 4) + warp, g_end = (t1 + kGroup - 1) >> 4;
    const int bs_mask = (1 << a.shift) - 1;
    const T* src = static_cast<const T*>(lane < 16 ? a.k : a.v) + kvh * a.head_stride;
    // the block of this lane's token of group g, or -1
    auto block_of = [&](int g) {
      const int t = g * kGroup + (lane & 15);
      return (g < g_end && t >= t0 && t < t1) ? table[t >> a.shift] : -1;
    };
    auto issue = [&](int g, int blk, int st) {
      const int t = g * kGroup + (lane & 15);
      const bool ok = blk >= 0 && blk < a.num_blocks;
      const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      if (lane == 0) {
        s_mask[warp][st] = mask;
        mbar_arrive_expect_tx(&bars[warp][st], __popc(mask) * 2 * D * (int)sizeof(T));
      }
      if (!ok && g < g_end && t >= t0 && t < t1) atomicOr(a.err_word, kErrBadBlock);
      __syncwarp();
      T* dst = ring + (st * 2 + (lane >> 4)) * S::kTile + (lane & 15) * S::kPitch;
      if (ok) {
        bulk_copy_g2s(dst, src + blk * a.block_stride + (t & bs_mask) * a.token_stride,
                      D * (int)sizeof(T), &bars[warp][st]);
      } else {  // zeros: a weight of 0 times whatever was there could be NaN
#pragma unroll
        for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    };
    int blk = block_of(g_first);
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) {
      const int g = g_first + st * kSplitWarps;
      const int next = block_of(g + kSplitWarps);
      if (g < g_end) issue(g, blk, st);
      blk = next;
    }
    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int g = g_first; g < g_end; g += kSplitWarps) {
      const int ahead = g + (kStages - 1) * kSplitWarps;
      const int next = block_of(ahead + kSplitWarps);
      if (ahead < g_end) issue(ahead, blk, st == 0 ? kStages - 1 : st - 1);
      blk = next;
      ok = mbar_wait_clocked(&bars[warp][st], phase);
      if (!ok) break;
      const uint32_t mask = s_mask[warp][st];
      const T* sk = ring + st * 2 * S::kTile;
      const T* sv = sk + S::kTile;
      float s[2][4] = {};
      {
        const int r = (lane & 7) + (lane >> 4) * 8, c = ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kf[4];
          ldsm_x4(kf, smem_addr(sk + r * S::kPitch + ks * 16 + c));
          Elem<T>::mma(s[0], qf[ks], kf[0], kf[1]);
          Elem<T>::mma(s[1], qf[ks], kf[2], kf[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] *= a.scale_log2;
      if (mask != 0xffffu || (g + 1) * kGroup > lo_lim) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = n * 8 + (lane & 3) * 2 + (j & 1);
            if (!((mask >> c) & 1) || g * kGroup + c >= lim[j >> 1]) s[n][j] = -INFINITY;
          }
      }
      uint32_t pf[4];
      float fix[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[h], mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        fix[h] = ex2_approx(m[h] - base);
        m[h] = mn;
        const float p0 = ex2_approx(s[0][2 * h] - base), p1 = ex2_approx(s[0][2 * h + 1] - base);
        const float p2 = ex2_approx(s[1][2 * h] - base), p3 = ex2_approx(s[1][2 * h + 1] - base);
        l[h] = l[h] * fix[h] + ((p0 + p1) + (p2 + p3));
        // the weights are rounded to the cache's type for the tensor cores (a
        // relative 2^-9 in bf16, 2^-12 in fp16, each its own way); their sum is not
        pf[h] = Elem<T>::pack(p0, p1);
        pf[h + 2] = Elem<T>::pack(p2, p3);
      }
      if (__any_sync(0xffffffffu, fix[0] != 1.f || fix[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= fix[0];
          o[i][1] *= fix[0];
          o[i][2] *= fix[1];
          o[i][3] *= fix[1];
        }
      }
      {
        const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = (lane >> 4) * 8;
#pragma unroll
        for (int dd = 0; dd < D / 16; ++dd) {
          uint32_t vf[4];
          ldsm_x4_t(vf, smem_addr(sv + r * S::kPitch + dd * 16 + c));
          Elem<T>::mma(o[2 * dd], pf, vf[0], vf[1]);
          Elem<T>::mma(o[2 * dd + 1], pf, vf[2], vf[3]);
        }
      }
      __syncwarp();
      if (++st == kStages) {
        st = 0;
        phase ^= 1;
      }
    }
    if (!ok) {
      // the copies in flight land before this CTA's shared memory goes to another
      for (int i = 0; i < kStages; ++i) mbar_wait_clocked(&bars[warp][i], phase, 200000000ll);
      atomicOr(a.err_word, kErrTimeout);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
  }

  // join the four warps
  float* so = reinterpret_cast<float*>(ring);
  if ((lane & 3) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s_m[warp][row0 + 8 * h] = m[h];
      s_l[warp][row0 + 8 * h] = l[h];
    }
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2*>(so + (row0 + 8 * h) * D + i * 8 + (lane & 3) * 2) =
          make_float2(o[i][2 * h], o[i][2 * h + 1]);
  __syncthreads();
  const int64_t rows_all = (int64_t)a.B * a.hq;
  const int64_t slab = (prefix ? split : a.prefix_splits + split) * rows_all;
  for (int i = tid; i < kRows * (D / 4); i += kSplitWarps * 32) {
    const int rr = i / (D / 4), c = (i % (D / 4)) * 4;
    const int r = tile * kRows + rr;
    if (r >= n_rows) break;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSplitWarps; ++w) mm = fmaxf(mm, s_m[w][rr]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kSplitWarps; ++w) {
      const float f = ex2_approx(s_m[w][rr] - base);
      ll += s_l[w][rr] * f;
      const float4 x = *reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(sq + S::kQElems + w * S::kWarpElems) + rr * D + c);
      acc.x += x.x * f;
      acc.y += x.y * f;
      acc.z += x.z * f;
      acc.w += x.w * f;
    }
    const int b = prefix ? r / a.G : b0, g = prefix ? r % a.G : r;
    const int64_t at = slab + (int64_t)b * a.hq + kvh * a.G + g;
    if (c == 0) a.part_ml[at] = make_float2(mm, ll);
    if (ll != 0.f) *reinterpret_cast<float4*>(a.part_o + at * D + c) = acc;
  }
}

// One warp to a query head: rescale the parts to their common maximum, sum,
// divide.  A part that holds nothing (sum 0) is not read; a NaN among the scores
// makes its part's sum NaN and so the row NaN.
template <typename T, int D>
__global__ void __launch_bounds__(128) join_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.B * a.hq;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int splits = a.prefix_splits + a.own_splits;
  float mx = -INFINITY;
  for (int s = lane; s < splits; s += 32) mx = fmaxf(mx, a.part_ml[s * rows + row].x);
  mx = warp_max(mx);
  constexpr int W = D / 32;
  float acc[W] = {};
  float l = 0.f;
  for (int s = 0; s < splits; ++s) {
    const float2 ml = a.part_ml[s * rows + row];
    if (ml.y == 0.f) continue;
    const float f = ex2_approx(ml.x - mx);
    l += ml.y * f;
    const float* o = a.part_o + (s * rows + row) * D + lane * W;
    if constexpr (W == 4) {
      const float4 x = *reinterpret_cast<const float4*>(o);
      acc[0] += x.x * f;
      acc[1] += x.y * f;
      acc[2] += x.z * f;
      acc[3] += x.w * f;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(o);
      acc[0] += x.x * f;
      acc[1] += x.y * f;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + row * D + lane * W);
#pragma unroll
  for (int i = 0; i < W / 2; ++i) out[i] = Elem<T>::pack(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[row] = l == 0.f ? -INFINITY : mx * kLn2 + logf(l);
}

template <typename T, int D>
cudaError_t launch_typed(const AttnArgs& a, cudaStream_t stream) {
  using S = SplitSmem<D>;
  cudaError_t e;
  if (a.prefix_mma &&
      (e = launch_prefix_mma(a, std::is_same<T, __half>::value ? VT_DTYPE_F16 : VT_DTYPE_BF16, D,
                             stream)) != cudaSuccess)
    return e;
  const int64_t units = (a.prefix_mma ? 0 : (int64_t)a.prefix_tiles * a.hkv * a.prefix_splits) +
                        (int64_t)a.own_tiles * a.hkv * a.B * a.own_splits;
  split_kernel<T, D><<<(unsigned)units, kSplitWarps * 32, S::kBytes, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.B * a.hq;
  join_kernel<T, D><<<(unsigned)((rows + 3) / 4), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_prefix_attention() {
  cudaError_t e;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(split_kernel<__nv_bfloat16, 64>, attr, SplitSmem<64>::kBytes)) ||
      (e = cudaFuncSetAttribute(split_kernel<__nv_bfloat16, 128>, attr, SplitSmem<128>::kBytes)) ||
      (e = cudaFuncSetAttribute(split_kernel<__half, 64>, attr, SplitSmem<64>::kBytes)) ||
      (e = cudaFuncSetAttribute(split_kernel<__half, 128>, attr, SplitSmem<128>::kBytes)))
    return e;
  return prepare_prefix_mma();
}

cudaError_t launch_prefix_attention(const AttnArgs& a, int dtype, int head_dim,
                                    cudaStream_t stream) {
  if (dtype == VT_DTYPE_BF16)
    return head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(a, stream)
                           : launch_typed<__nv_bfloat16, 64>(a, stream);
  return head_dim == 128 ? launch_typed<__half, 128>(a, stream)
                         : launch_typed<__half, 64>(a, stream);
}

}  // namespace vt
