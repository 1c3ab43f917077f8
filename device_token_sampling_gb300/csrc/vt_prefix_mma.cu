// vt_prefix_mma.cu -- the shared prefix on the 5th-generation tensor cores.
//
// The rows of a kv head, B * G query heads against one prefix, are a matrix
// product S = Q K^T, a softmax, and a product P V.  A CTA takes up to 256 rows
// (two tiles of 128) and one split of the prefix, 64 tokens at a step:
//   - the load warp brings K and V tiles of 128 tokens by TMA, block by block of
//     the cache, into two-stage rings of 128-byte-swizzled shared memory;
//   - a thread per tile issues its MMAs (one for both was bound by its own
//     instructions, 2900 cycles a step; with one each a step takes 1850): S_t = Q_t K^T into tensor memory, O_t += P_t V
//     with P_t read from tensor memory and V as it lies (token-major);
//   - a warpgroup per tile, one thread to a row, turns S into weights: running
//     maximum and sum in registers, P in the cache's type over the first columns
//     of its own S.
// Each tile has two S buffers, so that its next scores are made while it is at its
// exponentials: with one, scores, exponentials and product of a tile are one
// serial chain (85 us for 1024 rows of 8 kv heads against 16384 tokens, where two
// take 71).  A warp rescales its rows'
// accumulators only when one of their maxima has grown.  (To wait until it has
// grown by 2^8 saved 4 us of those 85, but then the largest weight is no longer
// exactly 1, and the rounding of the weights to bf16 costs 1.5e-3 of the result
// instead of 1.07e-3.)
// What bounds it: per 64 tokens and 256 rows 1024 cycles of the special function
// units and 1280 of the tensor cores (the scores read 48 KB of shared memory a
// tile, at 128 bytes a cycle), on the chain of exponentials and products of the two
// tiles that share an SM.  The 71 us (78 with unit_kernel reading beside it) are
// 68.7 GFLOP at 970 TFLOP/s, half the measured bf16 rate of 1936, and 128 of the
// 152 SMs; the others work on the requests' own tokens meanwhile.
#include <type_traits>

#include "vt_paged.h"
#include "vt_umma.cuh"

namespace vt {
namespace {

constexpr int kStep = 64;         // tokens of a step
constexpr int kKvStages = 2;
constexpr int kMmaThreads = 352;  // two softmax warpgroups, an MMA warp to each, the load warp
constexpr int kMmaWarp = 8, kLoadWarp = 10;
constexpr int kMaskRing = 8;      // tiles whose token masks are kept

template <int D>
struct MmaSmem {
  static constexpr int kHalf = kTileRows * 128;            // 128 rows of 64 elements
  static constexpr int kTile = (D / 64) * kHalf;           // bytes of a Q, K or V tile
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kTile;
  static constexpr int kV = kK + kKvStages * kTile;
  static constexpr int kBytes = kV + kKvStages * kTile + 1024;  // room to align to 1024
};

// tensor memory columns: two S buffers of each tile, then O of each tile; P lies
// over the first half of the S it was made from
template <int D>
struct Tmem {
  static constexpr int kO = 4 * kStep;
  static __device__ __forceinline__ uint32_t s(int t, int j) {
    return (uint32_t)((t * 2 + (j & 1)) * kStep);
  }
};

struct Bars {
  uint64_t k_full[kKvStages], k_empty[kKvStages], v_full[kKvStages], v_empty[kKvStages];
  // of each tile, by the parity of the step where a second step may begin before
  // the first is noticed
  uint64_t s_full[2][2], p_full[2][2], pv_done[2], o_done[2];
  uint64_t v_tail;  // the last V tile's rows past the end are zeros
  uint64_t drained[2];  // a tile's MMAs after a wait has run out
};

template <typename T, int D>
__global__ void __launch_bounds__(kMmaThreads, 1)
    prefix_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  using S = MmaSmem<D>;
  using TM = Tmem<D>;
  extern __shared__ unsigned char dyn[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_mask[kMaskRing][4];
  __shared__ int s_whole[kMaskRing];
  const int tid = threadIdx.x, lane = tid & 31;
  // (through a shuffle, so that the roles' control flow and addresses are known to
  // be the same in a warp: MMA operands live in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t base = (smem_addr(dyn) + 1023) & ~1023u;
  unsigned char* mem = dyn + (base - smem_addr(dyn));

  asm volatile("griddepcontrol.launch_dependents;");
  int u = blockIdx.x;
  const int kvh = u % a.hkv;
  u /= a.hkv;
  const int pairs = (a.prefix_tiles + 1) / 2;
  const int pair = u % pairs, split = u / pairs;
  const int n_rows = a.B * a.G;
  const bool two = pair * 2 + 1 < a.prefix_tiles;
  const int t0 = split * a.prefix_chunk, t1 = min(t0 + a.prefix_chunk, a.prefix_len);
  const int n_tiles = (t1 - t0 + kTileTokens - 1) / kTileTokens;
  const int n_steps = (t1 - t0 + kStep - 1) / kStep;
  // the split ends inside a block: what the copy brings from behind its end may be
  // anything, and a weight of 0 times NaN is NaN
  const int box = min(1 << a.shift, kTileTokens);  // tokens of a copy
  const bool ragged = t1 % box != 0;

  if (tid == 0) {
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.k_empty[i], two ? 2 : 1);  // (each tile's MMAs)
      mbar_init(&bars.v_empty[i], two ? 2 : 1);
    }
    mbar_init(&bars.v_tail, 1);
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.s_full[t][i], 1);
        mbar_init(&bars.p_full[t][i], kTileRows);
      }
      mbar_init(&bars.pv_done[t], 1);
      mbar_init(&bars.o_done[t], 1);
      mbar_init(&bars.drained[t], 1);
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp < kMmaWarp) {
    // Q into swizzled shared memory, negated where the scale is negative, while the
    // load warp begins; eight loads at once
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
    constexpr int kAhead = 8, kChunks = D / 8;
    const int all = (two ? 2 : 1) * kTileRows * kChunks;
#pragma unroll 1
    for (int i0 = tid; i0 < all; i0 += kMmaWarp * 32 * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int i = i0 + q * kMmaWarp * 32, c = i % kChunks;
        const int r = pair * 2 * kTileRows + i / kChunks;
        v[q] = make_uint4(0, 0, 0, 0);
        if (i < all && r < n_rows)
          v[q] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                 (int64_t)(r / a.G) * a.q_row +
                                                 (int64_t)(kvh * a.G + r % a.G) * a.q_head + c * 8);
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int i = i0 + q * kMmaWarp * 32, c = i % kChunks, row = i / kChunks;
        if (i >= all) break;
        v[q].x ^= flip, v[q].y ^= flip, v[q].z ^= flip, v[q].w ^= flip;
        const int in = row % kTileRows;
        *reinterpret_cast<uint4*>(mem + S::kQ + (row / kTileRows) * S::kTile +
                                  (c / 8) * S::kHalf + in * 128 + (((c & 7) ^ (in & 7)) << 4)) =
            v[q];
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  // Q is there: all but the load warp
  if (warp != kLoadWarp)
    asm volatile("bar.sync 1, %0;" ::"n"(kLoadWarp * 32) : "memory");
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  const long long limit = a.wait_cycles;
  bool ok = true;

  if (warp == kLoadWarp) {
    // ---- loads -----------------------------------------------------------------
    const int boxes = kTileTokens / box;
    int k_issued = 0, v_issued = 0;  // tiles
    for (int j = 0; j < n_tiles; ++j) {
      const int st = j % kKvStages, tok0 = t0 + j * kTileTokens;
      const uint32_t par = ((j / kKvStages) & 1) ^ 1;
      // the blocks of this tile, up to 128 of them: four a lane
      int blk[4];
      unsigned good[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = q * 32 + lane, tok = tok0 + i * box;
        blk[q] = i < boxes && tok < t1 ? a.prefix_blocks[tok >> a.shift] : -1;
        const bool fine = blk[q] >= 0 && blk[q] < a.num_blocks;
        if (i < boxes && tok < t1 && !fine) atomicOr(a.err_word, kErrBadBlock);
        if (!fine) blk[q] = a.num_blocks;  // outside: the copy fills zeros
        good[q] = __ballot_sync(0xffffffffu, fine);
      }
      if (lane < 4) {
        uint32_t m = 0;
        for (int i = 0; i < 32; ++i) {
          const int t = lane * 32 + i, bx = t / box;
          m |= ((good[bx >> 5] >> (bx & 31)) & 1u) && tok0 + t < t1 ? 1u << i : 0u;
        }
        s_mask[j % kMaskRing][lane] = m;
        const unsigned all = __ballot_sync(0xfu, m == 0xffffffffu);
        if (lane == 0) s_whole[j % kMaskRing] = all == 0xfu;
      }
      __syncwarp();
      const int in_block = tok0 & ((1 << a.shift) - 1);  // (blocks longer than a tile)
      ok = warp_wait(&bars.k_empty[st], par, limit);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&bars.k_full[st], S::kTile);
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = q * 32 + lane;
        if (i < boxes)
          for (int h = 0; h < D / 64; ++h)
            tma_tile(base + S::kK + st * S::kTile + h * S::kHalf + i * box * 128, &map_k,
                     &bars.k_full[st], h * 64, in_block, kvh, blk[q]);
      }
      k_issued = j + 1;
      ok = warp_wait(&bars.v_empty[st], par, limit);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&bars.v_full[st], S::kTile);
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = q * 32 + lane;
        if (i < boxes)
          for (int h = 0; h < D / 64; ++h)
            tma_tile(base + S::kV + st * S::kTile + h * S::kHalf + i * box * 128, &map_v,
                     &bars.v_full[st], h * 64, in_block, kvh, blk[q]);
      }
      v_issued = j + 1;
    }
    if (ragged && v_issued == n_tiles) {
      const int j = n_tiles - 1, st = j % kKvStages;
      ok = warp_wait(&bars.v_full[st], (j / kKvStages) & 1, limit);
      const int from = t1 - t0 - j * kTileTokens, to = (from + box - 1) / box * box;
      for (int i = from * 8 + lane; i < to * 8; i += 32)
        for (int h = 0; h < D / 64; ++h)
          *reinterpret_cast<uint4*>(mem + S::kV + st * S::kTile + h * S::kHalf + i * 16) =
              make_uint4(0, 0, 0, 0);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.v_tail);
    }
    // no copy is in flight when the CTA's memory goes to another
    for (int j = max(0, k_issued - kKvStages); j < k_issued; ++j)
      mbar_wait_clocked(&bars.k_full[j % kKvStages], (j / kKvStages) & 1, kDrainCycles);
    for (int j = max(0, v_issued - kKvStages); j < v_issued; ++j)
      mbar_wait_clocked(&bars.v_full[j % kKvStages], (j / kKvStages) & 1, kDrainCycles);
  } else if (warp >= kMmaWarp) {
    // ---- MMAs ------------------------------------------------------------------
    // The whole warp walks the steps and waits; one lane issues.
    constexpr uint32_t kType = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    // fp32 accumulators; K-major A and B; N = 64 tokens, M = 128
    constexpr uint32_t kIdescS = (1u << 4) | (kType << 7) | (kType << 10) |
                                 ((kStep / 8) << 17) | ((kTileRows / 16) << 24);
    // B (V) is N-major: its rows are tokens; N = D
    constexpr uint32_t kIdescO = (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) |
                                 ((uint32_t)(D / 8) << 17) | ((kTileRows / 16) << 24);
    constexpr uint32_t kHi = desc_hi(1024);
    const uint32_t q_lo = desc_lo(base + S::kQ, 16), k_lo = desc_lo(base + S::kK, 16),
                   v_lo = desc_lo(base + S::kV, S::kHalf);
    const int t = warp - kMmaWarp;
    const uint32_t a_lo = q_lo + t * (S::kTile >> 4), o = tmem + TM::kO + t * D;
    // step j is half j & 1 of tile j / 2, which is in stage (j / 2) & 1
    static_assert(kKvStages == 2, "stages by the parity of the tile");
    if (t == 0 || two) {
#pragma unroll 1
      for (int j = -1; j < n_steps; ++j) {
        const int n = j + 1, st_n = (n >> 1) & 1, st_j = (j >> 1) & 1;
        if (n < n_steps) {  // S_t = Q_t K^T of the next step
          if (!(n & 1)) ok = warp_wait(&bars.k_full[st_n], (n >> 2) & 1, limit);
          // the buffer is free when the product with its last P is done
          if (ok && j >= 1) ok = warp_wait(&bars.pv_done[t], (j - 1) & 1, limit);
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            const uint32_t d = tmem + TM::s(t, n),
                           b_lo = k_lo + st_n * (S::kTile >> 4) + (n & 1) * (kStep * 128 >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = ((ks / 4) * S::kHalf + (ks % 4) * 32) >> 4;
              mma_ss(d, a_lo + off, b_lo + off, kHi, kIdescS, ks > 0);
            }
            mma_commit(&bars.s_full[t][n & 1]);
            if ((n & 1) || n == n_steps - 1) mma_commit(&bars.k_empty[st_n]);
          }
          __syncwarp();
        }
        if (j >= 0) {  // O_t += P_t V of this one
          ok = warp_wait(&bars.p_full[t][j & 1], (j >> 1) & 1, limit);
          if (ok && !(j & 1)) {
            ok = warp_wait(&bars.v_full[st_j], (j >> 2) & 1, limit);
            if (ok && ragged && (j >> 1) == n_tiles - 1) ok = warp_wait(&bars.v_tail, 0, limit);
          }
          if (!ok) break;
          fence_after();
          if (elect_one()) {
            const uint32_t a_t = tmem + TM::s(t, j),
                           b_lo = v_lo + st_j * (S::kTile >> 4) + (j & 1) * (kStep * 128 >> 4);
#pragma unroll
            for (int ks = 0; ks < kStep / 16; ++ks)
              mma_ts(o, a_t + ks * 8, b_lo + (ks * 16 * 128 >> 4), kHi, kIdescO,
                     ks > 0 ? 1u : (uint32_t)(j > 0));
            mma_commit(&bars.pv_done[t]);
            if ((j & 1) || j == n_steps - 1) mma_commit(&bars.v_empty[st_j]);
            if (j == n_steps - 1) mma_commit(&bars.o_done[t]);
          }
          __syncwarp();
        }
      }
      if (!ok) {  // none of its MMAs is in flight when the CTA's memory goes to another
        if (elect_one()) mma_commit(&bars.drained[t]);
        __syncwarp();
        mbar_wait_clocked(&bars.drained[t], 0, kDrainCycles);
      }
    }
  } else {
    // ---- softmax: warpgroup t, one thread to a row --------------------------------
    const int t = warp >> 2;
    if (t == 0 || two) {
      const int in = tid & (kTileRows - 1);
      const int r = (pair * 2 + t) * kTileRows + in;
      const bool live = r < n_rows;
      const int b = live ? r / a.G : 0, head = kvh * a.G + (live ? r % a.G : 0);
      const int lim = live ? min(max(a.seq_lens[b], 0), a.prefix_len) : 0x7fffffff;
      const int lim_min = __reduce_min_sync(0xffffffffu, lim);
      // (a scale of 0 as one that leaves masked scores at -inf)
      const float sc = fmaxf(fabsf(a.scale_log2), 1e-30f);
      const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane (warp % 4) * 32
      const uint32_t to = tmem + lanes + TM::kO + t * D;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n_steps; ++j) {
        ok = wait_for(&bars.s_full[t][j & 1], (j >> 1) & 1, limit);
        if (!__all_sync(0xffffffffu, ok)) break;
        fence_after();
        const uint32_t ts = tmem + lanes + TM::s(t, j);
        uint32_t s[2][32];
        tmem_ld32(s[0], ts);
        tmem_ld32(s[1], ts + 32);
        tmem_wait_ld();
        loaded(s[0]);
        loaded(s[1]);
        const int tok0 = t0 + j * kStep, ring = (j >> 1) % kMaskRing;
        if (!s_whole[ring] || tok0 + kStep > lim_min) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t mask = s_mask[ring][(j & 1) * 2 + q];
            const int left = lim - tok0 - q * 32;
            const uint32_t keep =
                mask & (left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((keep >> i) & 1)) s[q][i] = 0xff800000u;
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 32; i += 2)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            mx[q] = fmaxf(mx[q], __uint_as_float(s[q & 1][i + (q >> 1)]));
        const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc);
        const bool grow = m_new > m;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2_approx(m - m_new) : 1.f;
          if (grow) m = m_new;
          l *= f;
          if (j > 0) {
            ok = wait_for(&bars.pv_done[t], (j - 1) & 1, limit);
            if (!__all_sync(0xffffffffu, ok)) break;
            fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(o, to + c);
              tmem_wait_ld();
              loaded(o);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st32(to + c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int e = 2 * i;
          const float p0 = ex2_approx(__fmaf_rn(__uint_as_float(s[e >> 5][e & 31]), sc, -off));
          const float p1 =
              ex2_approx(__fmaf_rn(__uint_as_float(s[e >> 5][(e & 31) + 1]), sc, -off));
          sum[(2 * i) & 3] += p0;
          sum[(2 * i + 1) & 3] += p1;
          // the weights are rounded to the cache's type for the tensor cores (a
          // relative 2^-9 in bf16, 2^-12 in fp16, each its own way); the sum is not
          p[i] = pack2<T>(p0, p1);
        }
        tmem_st32(ts, p);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        fence_before();
        mbar_arrive(&bars.p_full[t][j & 1]);
      }
      // the row's part
      if (ok) ok = wait_for(&bars.o_done[t], 0, limit);
      if (__all_sync(0xffffffffu, ok)) {
        fence_after();
        const int64_t at = (int64_t)split * a.B * a.hq + (int64_t)b * a.hq + head;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(o, to + c);
          tmem_wait_ld();
          loaded(o);
          if (live && l != 0.f)
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(a.part_o + at * D + c + i) =
                  make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
        if (live) a.part_ml[at] = make_float2(m, l);
      }
    }
  }
  if (!ok) atomicOr(a.err_word, kErrTimeout);
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

bool make_map(CUtensorMap* map, const AttnArgs& a, const void* cache, int dtype, int head_dim) {
  return cache_map(map, cache, dtype, head_dim, a.shift, a.hkv, a.num_blocks, a.block_stride,
                   a.token_stride, a.head_stride);
}

template <typename T, int D>
cudaError_t launch_typed(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                         cudaStream_t stream) {
  const int grid = (a.prefix_tiles + 1) / 2 * a.hkv * a.prefix_splits;
  prefix_kernel<T, D><<<grid, kMmaThreads, MmaSmem<D>::kBytes, stream>>>(a, mk, mv);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_prefix_mma() {
  cudaError_t e;
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(prefix_kernel<__nv_bfloat16, 64>, attr, MmaSmem<64>::kBytes)) ||
      (e = cudaFuncSetAttribute(prefix_kernel<__nv_bfloat16, 128>, attr, MmaSmem<128>::kBytes)) ||
      (e = cudaFuncSetAttribute(prefix_kernel<__half, 64>, attr, MmaSmem<64>::kBytes)) ||
      (e = cudaFuncSetAttribute(prefix_kernel<__half, 128>, attr, MmaSmem<128>::kBytes)))
    return e;
  // (all of it, so that units find room beside it)
  const auto carve = cudaFuncAttributePreferredSharedMemoryCarveout;
  if ((e = cudaFuncSetAttribute(prefix_kernel<__nv_bfloat16, 64>, carve, 100)) ||
      (e = cudaFuncSetAttribute(prefix_kernel<__nv_bfloat16, 128>, carve, 100)) ||
      (e = cudaFuncSetAttribute(prefix_kernel<__half, 64>, carve, 100)) ||
      (e = cudaFuncSetAttribute(prefix_kernel<__half, 128>, carve, 100)))
    return e;
  encode_tiled();  // the driver's entry point, looked up once
  return cudaSuccess;
}

bool prefix_mma_takes(const AttnArgs& a) {
  // (whole swizzle atoms, 8 tokens, to a copy)
  return a.shift >= 3 && cache_map_takes(a.block_stride, a.token_stride, a.head_stride);
}

cudaError_t launch_prefix_mma(const AttnArgs& a, int dtype, int head_dim, cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!make_map(&mk, a, a.k, dtype, head_dim) || !make_map(&mv, a, a.v, dtype, head_dim))
    return cudaErrorInvalidValue;
  if (dtype == VT_DTYPE_BF16)
    return head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(a, mk, mv, stream)
                           : launch_typed<__nv_bfloat16, 64>(a, mk, mv, stream);
  return head_dim == 128 ? launch_typed<__half, 128>(a, mk, mv, stream)
                         : launch_typed<__half, 64>(a, mk, mv, stream);
}

}  // namespace vt
