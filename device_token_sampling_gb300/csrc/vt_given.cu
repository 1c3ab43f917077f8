// vt_given.cu -- draws from given uniform numbers by inversion.
//
// For one row: z_j = fl(x_j * fl(1/T)), m = max z, w_j = exp(z_j - m).  The kept
// set is a prefix of the order (z descending, index ascending): min-p, then
// top-k, then top-p (exclusive prefix mass <= p * mass).  The draw of u is the
// first kept j, in vocabulary order, whose inclusive mass exceeds u * W, W the
// kept mass.
//
// Tokens are whole numbers decided by comparing sums of up to 2^20 masses, so
// masses are fixed-point integers: their sums are exact and the same in any
// order, and a mass is within 2.5e-10 of exp() in relative terms plus half a
// unit of the fixed point (mass_of).  A prefix of N random such errors moves a
// boundary by about 2.5e-10 / sqrt(N) of W, which puts the chance of a row's
// token differing from the exact one below 1e-5 even for a flat row.
//
// One thread-block cluster to a row.  Each CTA keeps its slice of the row in
// shared memory (one read of the logits); everything after that runs on chip,
// with the cluster's sums exchanged through distributed shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "vt_device.cuh"
#include "vt_kernels.h"
#include "vt_sampler.h"

namespace cg = cooperative_groups;

namespace vt {
namespace {

constexpr int kGivenThreads = 512;
constexpr int kGivenWarps = kGivenThreads / 32;
constexpr int kSeg = 512;           // elements a warp takes at a time, in vocabulary order
constexpr int kMaxSegs = 128;       // segments of a slice
constexpr int kSelBins = 2048;
constexpr int kLoadChunks = 8;
constexpr int kMaxIdx = 0x7fffffff;
constexpr uint32_t kLowestKey = 0x00800000u;  // ord_key(-FLT_MAX): every finite element

// 2^(-i/128) in units of 2^-31, from powers of 2^(-1/128).
struct MassTable {
  uint32_t v[128];
  constexpr MassTable() : v() {
    double x = 2147483648.0;
    for (int i = 0; i < 128; ++i) {
      v[i] = (uint32_t)(x + 0.5);
      x *= 0.99459942348363317565247768622217;
    }
  }
};
__constant__ MassTable c_mass_table = MassTable();

// exp(z - m) for z <= m in units of 2^-S, rounded to nearest.
//   z - m = dh + dl exactly (Knuth's TwoSum); t = -(dh + dl) log2(e) as th + tl
//   with an error below 2^-45; k = the multiple of 1/128 next to t, r = k - t in
//   [-1/256, 1/256], so that w = 2^-floor(k) * table[128 frac(k)] * 2^r and
//   2^r - 1 is a cubic within 2^-38, whose fp32 evaluation is off by 2^-33.
__device__ __forceinline__ uint64_t mass_of(float z, float m, int S, const uint32_t* table) {
  const float dh = __fsub_rn(z, m);
  const float bb = __fsub_rn(dh, z);
  const float aa = __fsub_rn(dh, bb);
  const float dl = __fadd_rn(__fsub_rn(z, aa), __fsub_rn(-m, bb));
  const float th = __fmul_rn(-dh, kLog2e);
  float tl = __fmaf_rn(-dh, kLog2e, -th);
  tl = __fmaf_rn(-dh, 1.92596299e-8f, tl);  // log2(e) - fl(log2(e))
  tl = __fmaf_rn(-dl, kLog2e, tl);
  if (!(th < 62.f)) return 0;  // -inf, or below half a unit
  const float magic = 12582912.f;  // 1.5 * 2^23: the integer next to 128 th in the low bits
  const float kb = __fmaf_rn(th, 128.f, magic);
  const int k = __float_as_int(kb) - __float_as_int(magic);
  const float r = __fsub_rn(__fmaf_rn(__fsub_rn(kb, magic), 0.0078125f, -th), tl);
  const float q = __fmul_rn(
      r, __fmaf_rn(r, __fmaf_rn(r, 0.0555041087f, 0.240226507f), 0.693147181f));
  const int qi = __float2int_rn(__fmul_rn(q, 0x1p38f));
  const uint32_t t = table[k & 127];
  const int64_t mant = ((int64_t)t << 31) + (((int64_t)(uint64_t)t * qi) >> 7);
  const int sh = 62 - S + (k >> 7);
  return sh > 62 ? 0ull : (uint64_t)((mant + (1ll << (sh - 1))) >> sh);
}

// floor(f * W) for 0 <= f < 1, exactly; f >= 1 gives W - 1, f <= 0 and NaN give 0.
__device__ __forceinline__ uint64_t part_of(uint64_t W, float f) {
  if (!(f > 0.f)) return 0;
  if (f >= 1.f) return W - 1;
  const uint32_t b = __float_as_uint(f);
  const int sh = 150 - (int)(b >> 23);
  if (sh >= 128) return 0;
  const uint64_t man = (b & 0x7fffffu) | 0x800000u;
  const uint64_t hi = __umul64hi(W, man), lo = W * man;
  return sh < 64 ? (hi << (64 - sh)) | (lo >> sh) : hi >> (sh - 64);
}

// The kept set: keys above `key`, and elements at it up to index `idx`.
struct Cut {
  uint32_t key;
  int idx;
  __device__ __forceinline__ bool keeps(uint32_t k, int j) const {
    return k > key || (k == key && j <= idx);
  }
};

// What a CTA shows the others of its cluster (each field written once between
// two cluster barriers).
struct Shown {
  float max;
  float expsum;
  uint64_t mass;
  int count;
  int index;
};

struct Found {
  int bin;
  uint32_t count;      // elements in the bin
  uint64_t above_n, above_w;
};

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
};
template <typename T>
__device__ __forceinline__ float elem(T x);
template <>
__device__ __forceinline__ float elem(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float elem(float x) { return x; }

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T, bool STAGED>
struct Slice {
  static constexpr int N = Vec<T>::N;
  static constexpr int kIters = kSeg / (32 * N);
  const T* data;   // shared memory (padded with -inf to whole segments) or the row itself
  int n;           // elements of this CTA (may be <= 0)
  int base;        // vocabulary index of the first
  bool vec;        // 16-byte loads from global memory

  // elements at + 0 .. N - 1 of the slice; -inf past its end
  __device__ __forceinline__ void load(int at, float (&x)[N]) const {
    if (STAGED) {
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(data + at), x);
    } else if (vec && at + N <= n) {
      Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(data + at)), x);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = at + i < n ? elem(data[at + i]) : -INFINITY;
    }
  }
  __device__ __forceinline__ int segs() const { return n > 0 ? (n + kSeg - 1) / kSeg : 0; }
};

struct Shared {
  Shown shown;
  Found found;
  int best;
  uint32_t table[128];
  float red_f[kGivenWarps];
  uint64_t red_w[kGivenWarps];
  uint32_t red_n[kGivenWarps];
  int red_i[kGivenWarps];
  uint64_t bars[kLoadChunks];
  uint64_t seg_w[kMaxSegs];   // masses of the segments, then their inclusive sums
  int seg_n[kMaxSegs];
  uint32_t hist_n[kSelBins];
  uint64_t hist_w[kSelBins];
};

// The row's boundary by radix selection on the order key, 11 + 11 + 10 bits.
//   MASS: elements are kept while the mass before them is <= target.
//   else: the first `target` of them are kept (1 <= target <= their number).
// Every CTA of the cluster returns the same cut.
template <typename T, bool STAGED, bool MASS>
__device__ Cut select(const Slice<T, STAGED>& sl, Shared& sh, cg::cluster_group& cluster, Cut cut,
                      float inv_t, float m, int S, uint64_t target) {
  using SL = Slice<T, STAGED>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster.num_blocks();
  uint32_t prefix = 0;
  uint64_t above_n = 0, above_w = 0;
  uint32_t ties = 0;
  constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll 1
  for (int level = 0; level < 3; ++level) {
    const int shift = kShift[level], bits = kBits[level], top = shift + bits;
    for (int i = tid; i < kSelBins; i += kGivenThreads) {
      sh.hist_n[i] = 0;
      sh.hist_w[i] = 0;
    }
    if (tid == 0) sh.best = -1;
    __syncthreads();
    for (int s = warp; s < sl.segs(); s += kGivenWarps) {
#pragma unroll 1
      for (int i = 0; i < SL::kIters; ++i) {
        const int at = s * kSeg + (i * 32 + lane) * SL::N;
        float x[SL::N];
        sl.load(at, x);
#pragma unroll
        for (int e = 0; e < SL::N; ++e) {
          const float z = __fmul_rn(x[e], inv_t);
          const uint32_t k = ord_key(z);
          if (!cut.keeps(k, sl.base + at + e)) continue;
          if (level > 0 && (k >> top) != prefix) continue;
          const uint32_t bin = (k >> shift) & ((1u << bits) - 1);
          atomicAdd(&sh.hist_n[bin], 1u);
          if (MASS) {
            const uint64_t w = mass_of(z, m, S, sh.table);
            if (w) atomicAdd((unsigned long long*)&sh.hist_w[bin], (unsigned long long)w);
          }
        }
      }
    }
    cluster.sync();
    // four bins to a thread, in descending order; sums over the cluster, then a scan
    uint32_t cn[4];
    uint64_t cw[4], tw = 0;
    uint32_t tn = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int bin = kSelBins - 1 - (tid * 4 + q);
      cn[q] = 0;
      cw[q] = 0;
      for (int r = 0; r < C; ++r) {
        const Shared* o = cluster.map_shared_rank(&sh, r);
        cn[q] += o->hist_n[bin];
        if (MASS) cw[q] += o->hist_w[bin];
      }
      tn += cn[q];
      tw += cw[q];
    }
    uint32_t in = tn;
    uint64_t iw = tw;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t pn = __shfl_up_sync(0xffffffffu, in, o);
      const uint64_t pw = __shfl_up_sync(0xffffffffu, iw, o);
      if (lane >= o) {
        in += pn;
        iw += pw;
      }
    }
    if (lane == 31) {
      sh.red_n[warp] = in;
      sh.red_w[warp] = iw;
    }
    __syncthreads();
    uint64_t bn = above_n + in - tn, bw = above_w + iw - tw;
    for (int i = 0; i < warp; ++i) {
      bn += sh.red_n[i];
      bw += sh.red_w[i];
    }
    uint64_t an = bn, aw = bw;
    int mine = -1;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool here = cn[q] > 0 && (MASS ? aw <= target : an < target);
      if (here) mine = tid * 4 + q;  // the last such bin holds the boundary
      an += cn[q];
      aw += cw[q];
    }
    if (mine >= 0) atomicMax(&sh.best, mine);
    __syncthreads();
    if (mine >= 0 && mine == sh.best) {
      an = bn;
      aw = bw;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (tid * 4 + q == mine) {
          sh.found.bin = kSelBins - 1 - mine;
          sh.found.count = cn[q];
          sh.found.above_n = an;
          sh.found.above_w = aw;
        }
        an += cn[q];
        aw += cw[q];
      }
    }
    cluster.sync();  // also: no CTA clears its bins while another reads them
    prefix = (prefix << bits) | (uint32_t)sh.found.bin;
    above_n = sh.found.above_n;
    above_w = sh.found.above_w;
    ties = sh.found.count;
  }
  const uint32_t key = prefix;
  uint64_t take;
  if (MASS) {
    const uint64_t w = mass_of(key_value(key), m, S, sh.table);
    take = w ? (target - above_w) / w + 1 : ties;
  } else {
    take = target - above_n;
  }
  const int old_idx = key == cut.key ? cut.idx : kMaxIdx;
  if (take >= ties) return Cut{key, old_idx};

  // the index of the take-th of the equal elements
  for (int s = warp; s < sl.segs(); s += kGivenWarps) {
    int c = 0;
#pragma unroll 1
    for (int i = 0; i < SL::kIters; ++i) {
      const int at = s * kSeg + (i * 32 + lane) * SL::N;
      float x[SL::N];
      sl.load(at, x);
#pragma unroll
      for (int e = 0; e < SL::N; ++e)
        c += ord_key(__fmul_rn(x[e], inv_t)) == key && sl.base + at + e <= old_idx;
    }
    c = warp_sum_i(c);
    if (lane == 0) sh.seg_n[s] = c;
  }
  __syncthreads();
  if (tid == 0) {
    int c = 0;
    for (int s = 0; s < sl.segs(); ++s) c += sh.seg_n[s];
    sh.shown.count = c;
    sh.shown.index = -1;
  }
  cluster.sync();
  uint64_t before = 0;
  for (int r = 0; r < (int)cluster.block_rank(); ++r)
    before += cluster.map_shared_rank(&sh, r)->shown.count;
  if (take > before && take <= before + sh.shown.count && warp == 0) {
    int left = (int)(take - before), s = 0;
    while (left > sh.seg_n[s]) left -= sh.seg_n[s++];
    for (int i = 0; i < SL::kIters; ++i) {
      const int at = s * kSeg + (i * 32 + lane) * SL::N;
      float x[SL::N];
      sl.load(at, x);
      int c = 0;
#pragma unroll
      for (int e = 0; e < SL::N; ++e)
        c += ord_key(__fmul_rn(x[e], inv_t)) == key && sl.base + at + e <= old_idx;
      int inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
      }
      if (left > inc - c && left <= inc) {
        int at_tie = left - (inc - c);
#pragma unroll
        for (int e = 0; e < SL::N; ++e)
          if (ord_key(__fmul_rn(x[e], inv_t)) == key && --at_tie == 0)
            sh.shown.index = sl.base + at + e;
      }
      left -= __shfl_sync(0xffffffffu, inc, 31);
      if (left <= 0) break;
    }
  }
  cluster.sync();
  int idx = -1;
  for (int r = 0; r < C; ++r) idx = max(idx, cluster.map_shared_rank(&sh, r)->shown.index);
  cluster.sync();
  return Cut{key, idx};
}

// Mass (and number) of the kept elements, by segment into sh.seg_w as inclusive
// sums; returns the cluster's total and, in *before, that of the CTAs ahead.
template <typename T, bool STAGED>
__device__ uint64_t kept_mass(const Slice<T, STAGED>& sl, Shared& sh, cg::cluster_group& cluster,
                              const Cut& cut, float inv_t, float m, int S, uint64_t* before) {
  using SL = Slice<T, STAGED>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int s = warp; s < sl.segs(); s += kGivenWarps) {
    uint64_t w = 0;
#pragma unroll 1
    for (int i = 0; i < SL::kIters; ++i) {
      const int at = s * kSeg + (i * 32 + lane) * SL::N;
      float x[SL::N];
      sl.load(at, x);
#pragma unroll
      for (int e = 0; e < SL::N; ++e) {
        const float z = __fmul_rn(x[e], inv_t);
        if (cut.keeps(ord_key(z), sl.base + at + e)) w += mass_of(z, m, S, sh.table);
      }
    }
    w = warp_sum_u64(w);
    if (lane == 0) sh.seg_w[s] = w;
  }
  __syncthreads();
  if (warp == 0) {
    uint64_t carry = 0;
    for (int s0 = 0; s0 < sl.segs(); s0 += 32) {
      uint64_t w = s0 + lane < sl.segs() ? sh.seg_w[s0 + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t p = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += p;
      }
      w += carry;
      if (s0 + lane < sl.segs()) sh.seg_w[s0 + lane] = w;
      carry = __shfl_sync(0xffffffffu, w, 31);
    }
    if (lane == 0) sh.shown.mass = carry;
  }
  cluster.sync();
  uint64_t total = 0, b = 0;
  for (int r = 0; r < (int)cluster.num_blocks(); ++r) {
    if (r == (int)cluster.block_rank()) b = total;
    total += cluster.map_shared_rank(&sh, r)->shown.mass;
  }
  cluster.sync();
  *before = b;
  return total;
}

// The first kept element of this CTA whose inclusive mass (from the CTA's start)
// exceeds t; one warp, t below the CTA's mass.
template <typename T, bool STAGED>
__device__ int find_draw(const Slice<T, STAGED>& sl, const Shared& sh, const Cut& cut, float inv_t,
                         float m, int S, uint64_t t, float* z_out) {
  using SL = Slice<T, STAGED>;
  const int lane = threadIdx.x & 31;
  int s = 0;
  for (int s0 = 0; s0 < sl.segs(); s0 += 32) {
    const bool past = s0 + lane < sl.segs() && sh.seg_w[s0 + lane] <= t;
    s += __popc(__ballot_sync(0xffffffffu, past));
  }
  if (s > 0) t -= sh.seg_w[s - 1];
  int idx = -1;
  float zz = 0.f;
  for (int i = 0; i < SL::kIters; ++i) {
    const int at = s * kSeg + (i * 32 + lane) * SL::N;
    float x[SL::N];
    sl.load(at, x);
    uint64_t w[SL::N], sum = 0;
#pragma unroll
    for (int e = 0; e < SL::N; ++e) {
      const float z = __fmul_rn(x[e], inv_t);
      w[e] = cut.keeps(ord_key(z), sl.base + at + e) ? mass_of(z, m, S, sh.table) : 0;
      sum += w[e];
    }
    uint64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t p = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += p;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, inc > t);
    if (hit) {
      const int owner = __ffs(hit) - 1;
      uint64_t run = inc - sum;
#pragma unroll
      for (int e = 0; e < SL::N; ++e) {
        run += w[e];
        if (idx < 0 && run > t) {
          idx = sl.base + at + e;
          zz = __fmul_rn(x[e], inv_t);
        }
      }
      *z_out = __shfl_sync(0xffffffffu, zz, owner);
      return __shfl_sync(0xffffffffu, idx, owner);
    }
    t -= __shfl_sync(0xffffffffu, inc, 31);
  }
  *z_out = 0.f;
  return -1;
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kGivenThreads) given_kernel(GivenArgs a) {
  using SL = Slice<T, STAGED>;
  extern __shared__ __align__(128) unsigned char dyn[];
  Shared& sh = *reinterpret_cast<Shared*>(dyn);
  T* stage = reinterpret_cast<T*>(dyn + ((sizeof(Shared) + 127) / 128) * 128);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int row = blockIdx.x / C;
  const RowParams P = a.params[row];
  const T* src = static_cast<const T*>(a.logits) + (int64_t)row * a.ld + (int64_t)rank * a.slice;
  SL sl;
  sl.base = rank * a.slice;
  sl.n = min(a.slice, a.V - sl.base);
  sl.vec = a.aligned;
  sl.data = STAGED ? stage : src;
  if (tid < 128) sh.table[tid] = c_mass_table.v[tid];

  // the row's maximum; with STAGED, taken as the slice arrives
  float mx = -INFINITY;
  const int n_pad = sl.segs() * kSeg;
  if (STAGED) {
    const int chunk = (((n_pad / kLoadChunks) + kSeg - 1) / kSeg) * kSeg;
    const int n_bulk = a.aligned && sl.n > 0 ? sl.n / SL::N * SL::N : 0;
    if (tid < kLoadChunks) mbar_init(&sh.bars[tid], 1);
    fence_mbar_init();
    __syncthreads();
    if (tid == 0 && n_bulk > 0) {
      for (int c = 0; c * chunk < n_bulk; ++c) {
        const uint32_t bytes = (uint32_t)min(chunk, n_bulk - c * chunk) * sizeof(T);
        mbar_arrive_expect_tx(&sh.bars[c], bytes);
        bulk_copy_g2s(stage + c * chunk, src + c * chunk, bytes, &sh.bars[c]);
      }
    }
    const T none = static_cast<T>(-INFINITY);
    for (int i = n_bulk + tid; i < n_pad; i += kGivenThreads) stage[i] = i < sl.n ? src[i] : none;
    __syncthreads();
    for (int c = 0; c * chunk < n_pad; ++c) {
      if (c * chunk < n_bulk && !mbar_wait_bounded(&sh.bars[c], 0)) atomicOr(a.err_word, kErrTimeout);
      const int end = min(n_pad, (c + 1) * chunk);
      for (int at = c * chunk + tid * SL::N; at < end; at += kGivenThreads * SL::N) {
        float x[SL::N];
        sl.load(at, x);
#pragma unroll
        for (int e = 0; e < SL::N; ++e) mx = max_nan(mx, x[e]);
      }
    }
  } else {
    for (int at = tid * SL::N; at < sl.n; at += kGivenThreads * SL::N) {
      float x[SL::N];
      sl.load(at, x);
#pragma unroll
      for (int e = 0; e < SL::N; ++e) mx = max_nan(mx, x[e]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) sh.red_f[warp] = mx;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kGivenWarps; ++i) mx = max_nan(mx, sh.red_f[i]);
    sh.shown.max = mx;
  }
  cluster.sync();
  mx = -INFINITY;
  for (int r = 0; r < C; ++r) mx = max_nan(mx, cluster.map_shared_rank(&sh, r)->shown.max);
  const float inv_t = P.inv_t;
  const float m = __fmul_rn(mx, inv_t);
  const int status = isnan(mx) || m == INFINITY ? kRowNonfinite : m == -INFINITY ? kRowEmpty : kRowOk;
  if (rank == 0 && tid == 0) a.row_status[row] = status;
  int32_t* out_tok = a.out_tokens + (int64_t)row * a.draws;
  float* out_lp = a.out_logprobs ? a.out_logprobs + (int64_t)row * a.draws : nullptr;
  if (status != kRowOk) {
    for (int d = rank * kGivenThreads + tid; d < a.draws; d += C * kGivenThreads) {
      out_tok[d] = -1;
      if (out_lp) out_lp[d] = NAN;
    }
    cluster.sync();  // the others have read this CTA's maximum
    return;
  }

  // ln sum exp(z - m) for the log-probs; a greedy row's lowest index at the maximum
  float expsum = 0.f;
  int first = kMaxIdx;
  const bool greedy = P.flags & kRowGreedy;
  if (out_lp || greedy) {
    for (int s = warp; s < sl.segs(); s += kGivenWarps) {
#pragma unroll 1
      for (int i = 0; i < SL::kIters; ++i) {
        const int at = s * kSeg + (i * 32 + lane) * SL::N;
        float x[SL::N];
        sl.load(at, x);
#pragma unroll
        for (int e = 0; e < SL::N; ++e) {
          expsum += ex2_approx(__fmul_rn(__fsub_rn(__fmul_rn(x[e], inv_t), m), kLog2e));
          if (greedy && x[e] == mx) first = min(first, sl.base + at + e);
        }
      }
    }
    expsum = warp_sum_f(expsum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
    __syncthreads();
    if (lane == 0) {
      sh.red_f[warp] = expsum;
      sh.red_i[warp] = first;
    }
    __syncthreads();
    if (tid == 0) {
      expsum = 0.f;
      for (int i = 0; i < kGivenWarps; ++i) {
        expsum += sh.red_f[i];
        first = min(first, sh.red_i[i]);
      }
      sh.shown.expsum = expsum;
      sh.shown.index = first;
    }
    cluster.sync();
    expsum = 0.f;
    for (int r = 0; r < C; ++r) {
      const Shared* o = cluster.map_shared_rank(&sh, r);
      expsum += o->shown.expsum;
      first = min(first, o->shown.index);
    }
    cluster.sync();
  }
  const float ln_s = logf(expsum);
  if (greedy) {
    for (int d = rank * kGivenThreads + tid; d < a.draws; d += C * kGivenThreads) {
      out_tok[d] = first;
      if (out_lp) out_lp[d] = -ln_s;
    }
    return;
  }

  // the kept set
  const int S = a.mass_bits;
  Cut cut{kLowestKey, kMaxIdx};
  if (P.flags & kRowMinP) {
    // the smallest z with z - m >= ln(min_p), both sides in double
    float zt = __double2float_rn((double)m + P.log_min_p);
    if ((double)zt - (double)m < P.log_min_p) {
      zt = nextafterf(zt, INFINITY);
    } else {
      const float below = nextafterf(zt, -INFINITY);
      if ((double)below - (double)m >= P.log_min_p) zt = below;
    }
    cut.key = max(cut.key, ord_key(zt));
  }
  if (P.top_k > 1 && P.top_k < a.V) {
    int c = 0;
    for (int s = warp; s < sl.segs(); s += kGivenWarps) {
#pragma unroll 1
      for (int i = 0; i < SL::kIters; ++i) {
        const int at = s * kSeg + (i * 32 + lane) * SL::N;
        float x[SL::N];
        sl.load(at, x);
#pragma unroll
        for (int e = 0; e < SL::N; ++e) c += ord_key(__fmul_rn(x[e], inv_t)) >= cut.key;
      }
    }
    c = warp_sum_i(c);
    if (lane == 0) sh.red_i[warp] = c;
    __syncthreads();
    if (tid == 0) {
      c = 0;
      for (int i = 0; i < kGivenWarps; ++i) c += sh.red_i[i];
      sh.shown.count = c;
    }
    cluster.sync();
    int n = 0;
    for (int r = 0; r < C; ++r) n += cluster.map_shared_rank(&sh, r)->shown.count;
    cluster.sync();
    if (n > P.top_k)
      cut = select<T, STAGED, false>(sl, sh, cluster, cut, inv_t, m, S, (uint64_t)P.top_k);
  }
  uint64_t before;
  uint64_t W = kept_mass(sl, sh, cluster, cut, inv_t, m, S, &before);
  if (P.flags & kRowTopP) {
    cut = select<T, STAGED, true>(sl, sh, cluster, cut, inv_t, m, S, part_of(W, P.top_p));
    W = kept_mass(sl, sh, cluster, cut, inv_t, m, S, &before);
  }

  // the draws: each by a warp of the CTA that holds its mass
  const uint64_t mine = sh.shown.mass;
  for (int d = warp; d < a.draws; d += kGivenWarps) {
    const uint64_t t = part_of(W, a.uniforms[(int64_t)row * a.draws + d]);
    if (t < before || t - before >= mine) continue;
    float z;
    const int j = find_draw(sl, sh, cut, inv_t, m, S, t - before, &z);
    if (lane == 0) {
      out_tok[d] = j;
      if (out_lp) out_lp[d] = __fsub_rn(__fsub_rn(z, m), ln_s);
    }
  }
}

template <typename T, bool STAGED>
cudaError_t launch_given_typed(const GivenArgs& a, int cluster, size_t smem, cudaStream_t stream) {
  auto* kernel = given_kernel<T, STAGED>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && cluster > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * cluster));
  cfg.blockDim = dim3(kGivenThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_given(GivenArgs a, int dtype, int num_sms, cudaStream_t stream) {
  const int es = dtype == VT_DTYPE_F32 ? 4 : 2;
  // slices small enough for two CTAs on an SM, and for few rows enough CTAs to
  // fill the GPU
  int cluster = 1;
  auto slice_of = [&](int c) { return ((a.V + c - 1) / c + kSeg - 1) / kSeg * kSeg; };
  while (cluster < 16 && ((int64_t)slice_of(cluster) * es > 80 * 1024 ||
                          slice_of(cluster) > kSeg * kMaxSegs ||
                          ((int64_t)a.B * cluster < 2 * num_sms && slice_of(cluster) > 4096)))
    cluster *= 2;
  a.slice = slice_of(cluster);
  // the largest scale whose sums of V masses stay below 2^63
  int bits = 0;
  while ((1ll << bits) < a.V) ++bits;
  a.mass_bits = min(45, 62 - bits);
  const size_t head = (sizeof(Shared) + 127) / 128 * 128;
  const size_t staged = head + (size_t)a.slice * es;
  const bool fits = staged <= 227 * 1024 - 1024;
  if (dtype == VT_DTYPE_F32)
    return fits ? launch_given_typed<float, true>(a, cluster, staged, stream)
                : launch_given_typed<float, false>(a, cluster, head, stream);
  return fits ? launch_given_typed<__nv_bfloat16, true>(a, cluster, staged, stream)
              : launch_given_typed<__nv_bfloat16, false>(a, cluster, head, stream);
}

}  // namespace vt
