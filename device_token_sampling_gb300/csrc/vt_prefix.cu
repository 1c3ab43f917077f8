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

constexpr int kGroup = 16;     // tokens a warp takes at a time
constexpr int kUnitWarps = 8;  // on an SM
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

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// 16 bytes global -> shared, zeros where !ok.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(ok ? 16 : 0)
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
struct UnitSmem {
  static constexpr int kPitch = D + 8;                      // elements: rows 16 bytes apart in banks
  static constexpr int kTile = kGroup * kPitch;             // elements of K (or V) of a group
  static constexpr size_t kBytes = 2 * (size_t)kStages * 2 * kTile;
};

// A unit of work: 8 or 16 query rows of one kv head against the tokens [t0, t1)
// of one table.
struct Unit {
  int kvh, tile, split, b;  // b < 0: the prefix, for the rows of all requests
  int t0, t1;
  const int32_t* table;
};

__device__ __forceinline__ Unit unit_of(const AttnArgs& a, int u) {
  Unit n;
  const int n_prefix = a.prefix_mma ? 0 : a.prefix_tiles * a.hkv * a.prefix_splits;
  if (u < n_prefix) {
    n.kvh = u % a.hkv;
    n.tile = (u / a.hkv) % a.prefix_tiles;
    n.split = u / (a.hkv * a.prefix_tiles);
    n.b = -1;
    n.table = a.prefix_blocks;
    n.t0 = n.split * a.prefix_chunk;
    n.t1 = min(n.t0 + a.prefix_chunk, a.prefix_len);
    return n;
  }
  u -= n_prefix;
  n.kvh = u % a.hkv;
  n.tile = (u / a.hkv) % a.own_tiles;
  n.b = (u / (a.hkv * a.own_tiles)) % a.B;
  n.split = u / (a.hkv * a.own_tiles * a.B);
  n.table = a.table + (int64_t)n.b * a.ld_table;
  const int len = min(max(a.seq_lens[n.b], 0), a.cols << a.shift);
  const int base = a.prefix_len & ~(kGroup - 1);
  // a longer request than the host reckoned with gets longer splits
  const int even = ((len - base + a.own_splits - 1) / a.own_splits + kGroup - 1) & ~(kGroup - 1);
  const int chunk = max(a.own_chunk, even);
  const int64_t lo = base + (int64_t)n.split * chunk;
  n.t0 = (int)(lo < a.prefix_len ? a.prefix_len : lo < len ? lo : len);
  n.t1 = (int)(lo + chunk < len ? lo + chunk : len);
  return n;
}

// Every warp, a CTA of its own, takes units off a common counter and runs them
// through its ring of copies, 16 tokens at a time, with its own running maxima and
// sums; the copies of the next unit are under way while the last groups of one are
// worked on, so that the stream of loads does not pause between units (with a CTA
// of four warps to a unit the waits at its two ends were a third of the time).
// Results do not depend on which warp takes a unit.  One warp (27 KB) finds room
// beside a CTA of prefix_kernel, which four do not: nearly half of the own tokens
// are read while the tensor cores work on the prefix (256 requests, 16,384 shared
// tokens and up to 1,024 of their own, head_dim 128: 169 us with CTAs of four
// warps, 165 so; 37 requests of head_dim 64, where four have room too, 27.8 and
// 29.8).
//
// The products are S^T = K Q^T and O^T = V^T P^T: the 16 tokens (or dims) fill the
// MMA's 16 rows and the query heads of a kv head only its 8 columns, NQ tiles of
// them, where Q K^T would pad 4 or 8 heads to 16 rows.  P^T is S^T's fragment moved
// by one transpose.  Tokens are copied 16 bytes a lane (a bulk copy a token would
// be issued lane by lane).  What bounds it: HBM, in pieces of 256 bytes, with two
// groups (16 KB at head_dim 128) in flight in each of 8 warps of an SM; 542 MB in
// 106 us with the join (5.1 TB/s; 4 warps 121 us, 6 108).
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(32) unit_kernel(AttnArgs a) {
  using S = UnitSmem<D>;
  constexpr int kRows = 8 * NQ;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ int4 s_group[kStages];  // number, mask of its tokens, unit, last
  __shared__ Unit s_unit[4];         // the units under way
  const int lane = threadIdx.x;
  T* ring = reinterpret_cast<T*>(dyn);
  const int n_units = (a.prefix_mma ? 0 : a.prefix_tiles * a.hkv * a.prefix_splits) +
                      a.own_tiles * a.hkv * a.B * a.own_splits;
  asm volatile("griddepcontrol.launch_dependents;");

  const int64_t rows_all = (int64_t)a.B * a.hq;
  // where row i of a unit is among the query heads of all requests, or -1
  auto row_of = [&](const Unit& n, int i) -> int64_t {
    const int r = n.tile * kRows + i;
    if (n.b < 0) {
      if (r >= a.B * a.G) return -1;
      return (int64_t)(r / a.G) * a.hq + n.kvh * a.G + r % a.G;
    }
    return r < a.G ? (int64_t)n.b * a.hq + n.kvh * a.G + r : -1;
  };
  auto slab_of = [&](const Unit& n) -> int64_t {
    return (n.b < 0 ? n.split : a.prefix_splits + n.split) * rows_all;
  };
  auto pop = [&]() {
    int u = 0;
    if (lane == 0) u = atomicAdd(a.work, 1);
    return u;  // (lane 0's)
  };

  // ---- the side that issues copies
  constexpr int kLanes = D / 8;              // lanes to a token
  constexpr int kPerCopy = 32 / kLanes;      // tokens to a copy instruction
  const int bs_mask = (1 << a.shift) - 1;
  Unit in{};
  int g = 0, g_end = 0, blk = -1;
  int n_in = 0;    // units taken
  int seq_in = 0;  // groups issued
  int waiting = pop();
  auto block_of = [&](int gg) {  // the block of token lane % 16 of group gg, or -1
    const int t = gg * kGroup + (lane & 15);
    return (gg < g_end && t >= in.t0 && t < in.t1) ? in.table[t >> a.shift] : -1;
  };
  auto next_unit = [&]() {
    for (;;) {
      const int u = __shfl_sync(0xffffffffu, waiting, 0);
      if (u >= n_units) {
        g = g_end = 0;
        return;
      }
      waiting = pop();
      in = unit_of(a, u);
      if (in.b < 0) {  // no row attends past the longest
        int lim = 0;
        if (lane < kRows && in.tile * kRows + lane < a.B * a.G)
          lim = max(a.seq_lens[(in.tile * kRows + lane) / a.G], 0);
        in.t1 = min(in.t1, __reduce_max_sync(0xffffffffu, lim));
      }
      if (in.t0 < in.t1) break;
      if (lane < kRows) {
        const int64_t row = row_of(in, lane);
        if (row >= 0) a.part_ml[slab_of(in) + row] = make_float2(-INFINITY, 0.f);
      }
    }
    g = in.t0 >> 4;
    g_end = (in.t1 + kGroup - 1) >> 4;
    if (lane == 0) s_unit[n_in & 3] = in;
    ++n_in;
    blk = block_of(g);
  };
  auto issue = [&]() {
    if (g < g_end) {
      const int st = seq_in % kStages;
      const int t = g * kGroup + (lane & 15);
      const bool fine = blk >= 0 && blk < a.num_blocks;
      const uint32_t mask = __ballot_sync(0xffffffffu, fine) & 0xffffu;
      if (!fine && t >= in.t0 && t < in.t1) atomicOr(a.err_word, kErrBadBlock);
      if (lane == 0) s_group[st] = make_int4(g, (int)mask, (n_in - 1) & 3, g + 1 == g_end);
      // where this lane's token begins in the cache
      const int64_t at = fine ? blk * a.block_stride + (t & bs_mask) * a.token_stride : 0;
      blk = block_of(g + 1);
      const int64_t col = in.kvh * a.head_stride + (lane % kLanes) * 8;
      const uint32_t dst = smem_addr(ring + st * 2 * S::kTile + (lane / kLanes) * S::kPitch +
                                     (lane % kLanes) * 8);
#pragma unroll
      for (int i = 0; i < kGroup / kPerCopy; ++i) {
        const int token = i * kPerCopy + lane / kLanes;
        const int64_t off = __shfl_sync(0xffffffffu, at, token) + col;
        const bool ok = (mask >> token) & 1;
        const uint32_t to = dst + i * kPerCopy * S::kPitch * (int)sizeof(T);
        copy16(to, static_cast<const T*>(a.k) + off, ok);
        copy16(to + S::kTile * (int)sizeof(T), static_cast<const T*>(a.v) + off, ok);
      }
      ++seq_in;
      if (++g == g_end) next_unit();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  next_unit();
#pragma unroll 1
  for (int st = 0; st < kStages - 1; ++st) issue();

  // ---- the side that works on them
  Unit n{};
  float o[NQ][D / 16][4];
  float m[NQ][2], l[NQ][2];
  int lim[NQ][2], lo_lim = 0, unit = -1;
  uint32_t qf[NQ][D / 16][2];
#pragma unroll 1
  for (int seq = 0; seq < seq_in; ++seq) {
    issue();
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const int st = seq % kStages;
    const int4 info = s_group[st];
    const int gg = info.x;
    const uint32_t mask = (uint32_t)info.y;
    if (unit != info.z) {  // the first group of a unit
      unit = info.z;
      n = s_unit[info.z];
      int lo = 0x7fffffff;
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t row = row_of(n, nq * 8 + (lane & 3) * 2 + h);
          lim[nq][h] = n.t1;
          if (n.b < 0 && row >= 0)
            lim[nq][h] = min(max(a.seq_lens[row / a.hq], 0), a.prefix_len);
          lo = min(lo, lim[nq][h]);
          m[nq][h] = -INFINITY;
          l[nq][h] = 0.f;
        }
        const int64_t row = row_of(n, nq * 8 + (lane >> 2)), r = max(row, (int64_t)0);
        const T* q = static_cast<const T*>(a.q) + (r / a.hq) * a.q_row + (r % a.hq) * a.q_head +
                     (lane & 3) * 2;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[nq][ks][i] =
                row >= 0 ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + i * 8) : 0u;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nq][i][j] = 0.f;
      }
      lo_lim = __reduce_min_sync(0xffffffffu, lo);
    }
    const T* sk = ring + st * 2 * S::kTile;
    const T* sv = sk + S::kTile;
    // two sums a tile: the chain of dependent MMAs is half as long
    float s[NQ][2][4] = {};
    {
      const uint32_t at = smem_addr(sk + ((lane & 7) + ((lane >> 3) & 1) * 8) * S::kPitch +
                                    (lane >> 4) * 8);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t kf[4];
        ldsm_x4(kf, at + ks * 32);
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
          Elem<T>::mma(s[nq][ks & 1], kf, qf[nq][ks][0], qf[nq][ks][1]);
      }
    }
    uint32_t pf[NQ][2];
    bool rescale = false;
    float fix[NQ][2];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      float z[4];  // tokens lane / 4 and 8 + lane / 4 of rows 2 (lane % 4) and the next
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = (s[nq][0][j] + s[nq][1][j]) * a.scale_log2;
      if (mask != 0xffffu || (gg + 1) * kGroup > lo_lim) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = (lane >> 2) + (j >> 1) * 8;
          if (!((mask >> c) & 1) || gg * kGroup + c >= lim[nq][j & 1]) z[j] = -INFINITY;
        }
      }
      float p[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = fmaxf(z[h], z[h + 2]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float mn = fmaxf(m[nq][h], mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        fix[nq][h] = ex2_approx(m[nq][h] - base);
        rescale |= mn != m[nq][h];
        m[nq][h] = mn;
        p[h] = ex2_approx(z[h] - base);
        p[h + 2] = ex2_approx(z[h + 2] - base);
        l[nq][h] = l[nq][h] * fix[nq][h] + (p[h] + p[h + 2]);
      }
      // the weights are rounded to the cache's type for the tensor cores (a
      // relative 2^-9 in bf16, 2^-12 in fp16, each its own way); their sum is not
      pf[nq][0] = transpose8(Elem<T>::pack(p[0], p[1]));
      pf[nq][1] = transpose8(Elem<T>::pack(p[2], p[3]));
    }
    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[nq][i][j] *= fix[nq][j & 1];
    }
    {
      const uint32_t at = smem_addr(sv + ((lane & 7) + (lane >> 4) * 8) * S::kPitch +
                                    ((lane >> 3) & 1) * 8);
#pragma unroll
      for (int dd = 0; dd < D / 16; ++dd) {
        uint32_t vf[4];
        ldsm_x4_t(vf, at + dd * 32);
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) Elem<T>::mma(o[nq][dd], vf, pf[nq][0], pf[nq][1]);
      }
    }
    if (info.w) {  // the last group: the rows' parts
      unit = -1;
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sum = l[nq][h];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          const int64_t row = row_of(n, nq * 8 + (lane & 3) * 2 + h);
          if (row < 0) continue;
          const int64_t at = slab_of(n) + row;
          if (lane < 4) a.part_ml[at] = make_float2(m[nq][h], sum);
          if (sum == 0.f) continue;
          float* to = a.part_o + at * D + (lane >> 2);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            to[i * 16] = o[nq][i][h];
            to[i * 16 + 8] = o[nq][i][h + 2];
          }
        }
    }
    __syncwarp();
  }
  // (this grid's end then also means that of prefix_kernel, which it may overtake)
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One query head over the first `len` tokens of the prefix, token by token in fp32:
// the way of last resort of join_kernel.  One warp; a lane has D / 32 neighbouring
// elements.
template <typename T, int D>
__device__ __forceinline__ void attend_row(const AttnArgs& a, int64_t row, int len,
                                           float (&acc)[D / 32], float* max_out, float* sum_out) {
  constexpr int W = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t b = row / a.hq, head = row % a.hq;
  auto load = [&](const void* from, int64_t at, float (&x)[W]) {
    const T* p = static_cast<const T*>(from) + at + lane * W;
#pragma unroll
    for (int w = 0; w < W; ++w) x[w] = static_cast<float>(p[w]);
  };
  float q[W], m = -INFINITY, l = 0.f;
  load(a.q, b * a.q_row + head * a.q_head, q);
#pragma unroll
  for (int w = 0; w < W; ++w) acc[w] = 0.f;
#pragma unroll 1
  for (int t = 0; t < len; ++t) {
    const int blk = a.prefix_blocks[t >> a.shift];
    if (blk < 0 || blk >= a.num_blocks) continue;
    const int64_t at = blk * a.block_stride + (t & ((1 << a.shift) - 1)) * a.token_stride +
                       head / a.G * a.head_stride;
    float k[W], v[W], s = 0.f;
    load(a.k, at, k);
    load(a.v, at, v);
#pragma unroll
    for (int w = 0; w < W; ++w) s += q[w] * k[w];
    const float z = warp_sum_f(s) * a.scale_log2;
    const float mn = fmaxf(m, z), base = mn == -INFINITY ? 0.f : mn;
    const float f = ex2_approx(m - base), p = ex2_approx(z - base);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int w = 0; w < W; ++w) acc[w] = acc[w] * f + p * v[w];
  }
  *max_out = m;
  *sum_out = l;
}

// One warp to a query head: rescale the parts to their common maximum, sum,
// divide.  A part that holds nothing (sum 0) is not read; a NaN among the scores
// makes its part's sum NaN and so the row NaN.  The parts' factors are made a lane
// to a part and four parts are read at a time: one after another, the 21 parts of
// 64 requests behind 8,192 tokens cost 2 us more (52.3 and 50.2 over all), the 17
// of 37 requests 4 us (28.5 and 24.2).  What bounds it: those reads' latency.
//
// A request shorter than the prefix shares tiles of V with requests that attend to
// more of it.  Its weights there are 0, but 0 times an infinity or a NaN is NaN; a
// row of such a request that comes out NaN is made again from its own tokens alone.
// (Held to the 32 registers that it takes without that, this kernel spills: 64
// requests 47.5 us over all instead of 45.5.)
template <typename T, int D>
__global__ void __launch_bounds__(128) join_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.B * a.hq;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.work = 0;  // for the next call
  if (row >= rows) return;
  const int splits = a.prefix_splits + a.own_splits;
  float mx = -INFINITY;
  for (int s = lane; s < splits; s += 32) mx = fmaxf(mx, a.part_ml[s * rows + row].x);
  mx = warp_max(mx);
  constexpr int W = D / 32;
  constexpr int kAhead = 4;  // parts read at a time
  float acc[W] = {};
  float l = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < splits; s0 += 32) {  // a lane's part of these: its sum and factor
    const float2 ml = s0 + lane < splits ? a.part_ml[(s0 + lane) * rows + row]
                                         : make_float2(-INFINITY, 0.f);
    const bool some = ml.y != 0.f;
    const float f = some ? ex2_approx(ml.x - mx) : 0.f;
    if (some) l += ml.y * f;
    const unsigned full = __ballot_sync(0xffffffffu, some);
#pragma unroll 1
    for (int s = 0; s < 32 && full >> s; s += kAhead) {
      float x[kAhead][W];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {  // (in place of an empty part the first full one)
        const int part = s0 + ((full >> (s + k)) & 1 ? s + k : __ffs(full) - 1);
        const float* o = a.part_o + (part * rows + row) * D + lane * W;
        if constexpr (W == 4) {
          const float4 v = *reinterpret_cast<const float4*>(o);
          x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(o);
          x[k][0] = v.x, x[k][1] = v.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, s + k);
        if ((full >> (s + k)) & 1) {
#pragma unroll
          for (int w = 0; w < W; ++w) acc[w] += x[k][w] * fk;
        }
      }
    }
  }
  l = warp_sum_f(l);
  bool nan = false;
#pragma unroll
  for (int w = 0; w < W; ++w) nan |= acc[w] != acc[w];
  if (a.prefix_len > 0 && __any_sync(0xffffffffu, nan)) {
    const int len = max(a.seq_lens[row / a.hq], 0);
    if (len < a.prefix_len) attend_row<T, D>(a, row, len, acc, &mx, &l);
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
  using S = UnitSmem<D>;
  cudaError_t e;
  if (a.prefix_mma &&
      (e = launch_prefix_mma(a, std::is_same<T, __half>::value ? VT_DTYPE_F16 : VT_DTYPE_BF16, D,
                             stream)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.stream = stream;
  // beside prefix_kernel as its SMs get free; not before the work in front of that
  cfg.numAttrs = a.prefix_mma ? 1 : 0;
  const int64_t units = (a.prefix_mma ? 0 : (int64_t)a.prefix_tiles * a.hkv * a.prefix_splits) +
                        (int64_t)a.own_tiles * a.hkv * a.B * a.own_splits;
  const int64_t most = (int64_t)kUnitWarps * a.num_sms;
  cfg.gridDim = dim3((unsigned)(units < most ? units : most));
  cfg.blockDim = dim3(32);
  cfg.dynamicSmemBytes = S::kBytes;
  e = a.unit_rows == 8 ? cudaLaunchKernelEx(&cfg, unit_kernel<T, D, 1>, a)
                       : cudaLaunchKernelEx(&cfg, unit_kernel<T, D, 2>, a);
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  const int64_t rows = (int64_t)a.B * a.hq;
  cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, join_kernel<T, D>, a);
  // (join_kernel would have set the counter back)
  if (e != cudaSuccess) cudaMemsetAsync(a.work, 0, sizeof(int32_t), stream);
  return e;
}

}  // namespace

template <typename T, int D>
static cudaError_t prepare_units() {
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  // (the same division of an SM's memory as prefix_kernel's, to run beside it)
  const auto carve = cudaFuncAttributePreferredSharedMemoryCarveout;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(unit_kernel<T, D, 1>, attr, UnitSmem<D>::kBytes)) ||
      (e = cudaFuncSetAttribute(unit_kernel<T, D, 2>, attr, UnitSmem<D>::kBytes)) ||
      (e = cudaFuncSetAttribute(unit_kernel<T, D, 1>, carve, 100)) ||
      (e = cudaFuncSetAttribute(unit_kernel<T, D, 2>, carve, 100)))
    return e;
  return cudaSuccess;
}

cudaError_t prepare_prefix_attention() {
  cudaError_t e;
  if ((e = prepare_units<__nv_bfloat16, 64>()) || (e = prepare_units<__nv_bfloat16, 128>()) ||
      (e = prepare_units<__half, 64>()) || (e = prepare_units<__half, 128>()))
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
