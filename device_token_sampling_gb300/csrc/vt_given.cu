// vt_given.cu -- draws from given uniform numbers by inversion.
//
// For one row: z_j = fl(x_j * fl(1/T)), m = max z, w_j = exp(z_j - m).  The kept
// set is a prefix of the order (z descending, index ascending): min-p, then
// top-k, then top-p (exclusive prefix mass <= p * mass).  The draw of u is the
// first kept j, in vocabulary order, whose inclusive mass exceeds u * W, W the
// kept mass.
//
// Tokens are whole numbers decided by comparing sums of up to 2^20 masses, so
// masses are integers (struct Mass): their sums are exact and the same in any
// order, and a mass is within 6e-10 (rms 2e-10) of exp() in relative terms.  A
// prefix of N such errors moves a boundary by about 2e-10 / sqrt(N) of W (N the
// distinct values among bf16 logits), which puts the chance of a draw differing
// from the exact one below 1e-5 even for a flat row.
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
constexpr int kMaxCtas = 16;        // CTAs of a row at most
constexpr int kBins = 2048;
constexpr float kBinsPerNat = 64.f;  // linear bins: 32 nats below the maximum, then one for all
constexpr int kList = 2048;         // candidates a row's leader CTA holds
constexpr int kListTopK = 1024;     // largest top-k taken from group maxima
constexpr int kListPerThread = kList / kGivenThreads;
constexpr int kLoadChunks = 8;
constexpr int kMaxIdx = 0x7fffffff;

// 2^(i/128) in units of 2^-30, from powers of 2^(1/128).
struct MassTable {
  uint32_t v[128];
  constexpr MassTable() : v() {
    double x = 1073741824.0;
    for (int i = 0; i < 128; ++i) {
      v[i] = (uint32_t)(x + 0.5);
      x *= 1.0054299011128028;
    }
  }
};
__constant__ MassTable c_mass_table = MassTable();

constexpr int kElemBits = 53;  // masses of single elements: units of 2^-53 of 2^E

// Masses as integers: exp(z) = 2^(z log2(e)) relative to 2^E, the power of two
// next above the maximum, so that no subtraction of the maximum rounds.
//   p + e = z log2(e) with an error below 2^-40; k = the multiple of 1/128 next
//   to p, r = p - k + e in [-1/256, 1/256]: the mass is 2^floor(k) *
//   table[128 frac(k)] * 2^r, and 2^r - 1 is a cubic within 2^-38 whose fp32
//   evaluation is off by 2^-33.
// About 25 instructions, no division, one conversion and one shared load.  For a
// maximum beyond 2^13 the reduction would run out of bits; there z - m is
// exact wherever the mass is not 0 (z within a factor 2 of m), so the row's
// values are shifted by c = m (else c = 0).
struct Mass {
  float inv_t, c, floor_p;
  int e128;  // 128 * E
  const uint32_t* table;

  __device__ __forceinline__ Mass(float inv_t_, float m, const uint32_t* table_) {
    inv_t = inv_t_;
    table = table_;
    c = fabsf(m) < 8192.f ? 0.f : m;
    const int E = (int)floorf(__fmul_rn(m - c, kLog2e)) + 1;
    e128 = E * 128;
    floor_p = (float)(E - 62);
  }
  __device__ __forceinline__ float z(float x) const { return __fmul_rn(x, inv_t); }
  // mass of the tempered value z in units of 2^(E - kElemBits), truncated
  __device__ __forceinline__ uint64_t of(float z) const {
    z = __fsub_rn(z, c);
    const float p = fmaxf(__fmul_rn(z, kLog2e), floor_p);  // -inf and far below: mass 0
    const float e = __fmaf_rn(z, 1.92596303e-8f, __fmaf_rn(z, kLog2e, -p));
    const float magic = 12582912.f;  // 1.5 * 2^23: the integer next to 128 p in the low bits
    const float kb = __fmaf_rn(p, 128.f, magic);
    const int k = __float_as_int(kb) - __float_as_int(magic);
    const float r = __fadd_rn(__fmaf_rn(__fsub_rn(kb, magic), -0.0078125f, p), e);
    const float q = __fmul_rn(r, __fmaf_rn(r, __fmaf_rn(r, 238388332.f, 1031764991.f),
                                           2977044472.f));  // (2^r - 1) 2^32
    const int sh = 62 - kElemBits + ((e128 - k + 127) >> 7);
    const int64_t t = (int64_t)table[k & 127];
    const int64_t mant = (t << 32) + t * (int64_t)__float2int_rn(q);
    return p == floor_p ? 0ull : (uint64_t)mant >> sh;
  }
  // ln of a sum of masses in units of 2^(E - bits), relative to the maximum m
  __device__ __forceinline__ float ln_sum(uint64_t w, int bits, float m) const {
    const float E = (float)(e128 >> 7);
    const float lw = logf(__ull2float_rn(w) * exp2f((float)-bits));
    // E ln 2 - (m - c) in one rounding, ln 2 in two parts
    return lw + (__fmaf_rn(E, 0.693147182464599609375f, -__fsub_rn(m, c)) +
                 E * -1.904654299957e-9f);
  }
};

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

// The kept set: tempered values above z, and those at z up to index idx.
struct Cut {
  float z;
  int idx;
  __device__ __forceinline__ bool keeps(float v, int j) const {
    return v >= z && (idx == kMaxIdx || v > z || j <= idx);
  }
};

// A CTA's mailboxes: slot r is written by CTA r of its cluster before a cluster
// barrier and read here after it, so that no reader waits on remote loads.  Each
// field serves one exchange, or exchanges with another barrier between the
// reading of one and the writing of the next.
struct Mail {
  float max[kMaxCtas];
  float expsum[kMaxCtas];
  uint64_t mass[kMaxCtas], all[kMaxCtas], kept[kMaxCtas];
  int count[kMaxCtas], total[kMaxCtas];
  int index[kMaxCtas], tie[kMaxCtas];
  Cut cut;  // from the leader
  int ok;
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

// Inclusive sums over a warp.
template <typename U>
__device__ __forceinline__ U warp_scan(U v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const U p = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += p;
  }
  return v;
}

static_assert(2 * kListTopK <= kBins, "the groups' maxima fit their array");

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
  // position of the first of a lane's N elements in iteration i of segment s
  static __device__ __forceinline__ int at(int s, int i) {
    return s * kSeg + (i * 32 + (threadIdx.x & 31)) * N;
  }
};

// The candidates of a row in vocabulary order, on its leader CTA.
struct List {
  uint32_t key[kList];  // ord_key of the tempered value
  int idx[kList];
};

struct Hist {
  uint32_t own[kBins];
  union {
    uint32_t sum[kBins];     // over the cluster
    float group_max[kBins];  // maxima of groups of elements, of all CTAs
  };
};

struct Shared {
  Mail mail;
  float red_f[kGivenWarps];
  uint64_t red_w[kGivenWarps], red_n[kGivenWarps];
  int red_i[kGivenWarps];
  uint64_t bars[kLoadChunks];
  uint32_t table[128];
  uint64_t seg_w[kMaxSegs];   // masses of the segments, then their inclusive sums
  int seg_n[kMaxSegs];        // candidates of the segments, then those before each
  int lo, hi;
  int bin;
  uint32_t bin_n;
  uint64_t above;
  uint32_t digit_n[256];      // radix selection, 8 bits at a time
  unsigned long long digit_w[256];
  uint64_t run[kGivenThreads];  // inclusive masses of the threads' list entries
  union {
    Hist hist;
    List list;
  };
};

// The row of this cluster.
template <typename T, bool STAGED>
struct Row {
  Slice<T, STAGED> sl;
  Shared& sh;
  Mass mass;
  float m;        // tempered maximum
  int slice;      // elements per CTA
  int drop;       // row sums are in units of 2^(E - kElemBits + drop)
  __device__ __forceinline__ Row(const Slice<T, STAGED>& sl_, Shared& sh_, const Mass& mass_,
                                 float m_, int slice_, int drop_)
      : sl(sl_), sh(sh_), mass(mass_), m(m_), slice(slice_),
        drop(drop_) {}
  __device__ __forceinline__ Shared* at(int rank) {
    return cg::this_cluster().map_shared_rank(&sh, rank);
  }
  // thread r of the block stores v in this CTA's slot of CTA r's mailbox
  template <typename V>
  __device__ __forceinline__ void send(V (Mail::*field)[kMaxCtas], V v) {
    const int C = cg::this_cluster().num_blocks();
    if ((int)threadIdx.x < C)
      (at((int)threadIdx.x)->mail.*field)[cg::this_cluster().block_rank()] = v;
  }
  __device__ __forceinline__ uint64_t coarse(uint64_t w) const {
    return (w + (1ull << (drop - 1))) >> drop;
  }
  __device__ __forceinline__ float bins_below(float z) const {
    return __fmul_rn(__fsub_rn(m, z), kBinsPerNat);
  }
};

__device__ __forceinline__ int bin_of(float t) {
  return t < (float)(kBins - 1) ? (int)t : kBins - 1;
}

// Block-wide exclusive sum in thread order, and the total.
__device__ __forceinline__ uint64_t block_scan(Shared& sh, uint64_t w, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t inc = warp_scan(w);
  __syncthreads();
  if (lane == 31) sh.red_w[warp] = inc;
  __syncthreads();
  uint64_t before = inc - w, all = 0;
#pragma unroll
  for (int i = 0; i < kGivenWarps; ++i) {
    if (i < warp) before += sh.red_w[i];
    all += sh.red_w[i];
  }
  *total = all;
  return before;
}

// Sum over the block, in warp 0's order; every thread gets it.
__device__ __forceinline__ float block_sum(Shared& sh, float v) {
  v = warp_sum_f(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.red_f[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kGivenWarps; ++i) v += sh.red_f[i];
  return v;
}
__device__ __forceinline__ int block_sum(Shared& sh, int v) {
  v = warp_sum_i(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.red_i[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kGivenWarps; ++i) v += sh.red_i[i];
  return v;
}

// Of 256 digits' (elements, weight), counted from 255 down after `before`: the
// digit that holds the boundary, into sh.bin / bin_n / above.  Warp 0.
template <bool MASS>
__device__ __forceinline__ void find_digit(Shared& sh, uint64_t before, uint64_t target) {
  const int lane = threadIdx.x & 31;
  uint64_t v[8], sum = 0;
  uint32_t c[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    c[q] = sh.digit_n[255 - 8 * lane - q];
    v[q] = MASS ? (uint64_t)sh.digit_w[255 - 8 * lane - q] : c[q];
    sum += v[q];
  }
  uint64_t a = before + warp_scan(sum) - sum;
  int mine = -1;
  uint64_t mine_a = 0;
  uint32_t mine_c = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (c[q] > 0 && (MASS ? a <= target : a < target)) {
      mine = 8 * lane + q;
      mine_a = a;
      mine_c = c[q];
    }
    a += v[q];
  }
  const unsigned has = __ballot_sync(0xffffffffu, mine >= 0);
  if (has && lane == 31 - __clz(has)) {  // the last such digit
    sh.bin = 255 - mine;
    sh.bin_n = mine_c;
    sh.above = mine_a;
  }
}

// The row's boundary by radix selection on the order key, 8 bits at a time, for
// any number of equal elements.  The way of last resort: it counts every element
// by shared atomics, thousands to an address.
//   MASS: elements are kept while the mass before them is <= target.
//   else: the first `target` of them are kept (1 <= target <= their number).
// Every CTA of the cluster returns the same cut.
template <typename T, bool STAGED, bool MASS>
__device__ __noinline__ Cut radix_select(const Row<T, STAGED>& row_in, Cut cut, uint64_t target) {
  Row<T, STAGED> rw = row_in;  // in registers
  using SL = Slice<T, STAGED>;
  const SL& sl = rw.sl;
  Shared& sh = rw.sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster.block_rank();
  uint32_t prefix = 0;
  uint64_t before = 0;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) {
      sh.digit_n[tid] = 0;
      sh.digit_w[tid] = 0;
    }
    cluster.sync();
    for (int s = warp; s < sl.segs(); s += kGivenWarps) {
#pragma unroll 1
      for (int i = 0; i < SL::kIters; ++i) {
        const int at = SL::at(s, i);
        float x[SL::N];
        sl.load(at, x);
#pragma unroll
        for (int e = 0; e < SL::N; ++e) {
          const float z = rw.mass.z(x[e]);
          const uint32_t k = ord_key(z);
          if (!cut.keeps(z, sl.base + at + e)) continue;
          if (shift < 24 && (k >> (shift + 8)) != prefix) continue;
          const int bin = (k >> shift) & 255;
          atomicAdd(&sh.digit_n[bin], 1u);
          if (MASS) {
            const uint64_t w = rw.coarse(rw.mass.of(z));
            if (w) atomicAdd(&sh.digit_w[bin], (unsigned long long)w);
          }
        }
      }
    }
    __syncthreads();
    // the others' digits are added to the leader's, which finds the boundary
    if (rank != 0 && tid < 256 && sh.digit_n[tid]) {
      atomicAdd(&rw.at(0)->digit_n[tid], sh.digit_n[tid]);
      if (MASS) atomicAdd(&rw.at(0)->digit_w[tid], sh.digit_w[tid]);
    }
    cluster.sync();
    if (rank == 0 && warp == 0) find_digit<MASS>(sh, before, target);
    cluster.sync();
    const Shared* lead = rw.at(0);
    prefix = (prefix << 8) | (uint32_t)lead->bin;
    before = lead->above;
  }
  const uint32_t ties = rw.at(0)->bin_n;
  cluster.sync();
  const float zk = key_value(prefix);
  uint64_t take;
  if (MASS) {
    const uint64_t w = rw.coarse(rw.mass.of(zk));
    take = w ? (target - before) / w + 1 : ties;
  } else {
    take = target - before;
  }
  const int old_idx = zk == cut.z ? cut.idx : kMaxIdx;
  if (take >= ties) return Cut{zk, old_idx};

  // the index of the take-th of the equal elements
  int mine = 0;
  for (int s = warp; s < sl.segs(); s += kGivenWarps) {
    int c = 0;
#pragma unroll 1
    for (int i = 0; i < SL::kIters; ++i) {
      const int at = SL::at(s, i);
      float x[SL::N];
      sl.load(at, x);
#pragma unroll
      for (int e = 0; e < SL::N; ++e)
        c += rw.mass.z(x[e]) == zk && sl.base + at + e <= old_idx;
    }
    c = warp_sum_i(c);
    if (lane == 0) {
      sh.seg_n[s] = c;
      mine += c;
    }
  }
  mine = block_sum(sh, mine);
  rw.send(&Mail::total, mine);
  cluster.sync();
  uint64_t ahead = 0;
  for (int r = 0; r < rank; ++r) ahead += sh.mail.total[r];
  if (tid == 0) sh.lo = -1;
  __syncthreads();
  if (take > ahead && take <= ahead + mine && warp == 0) {
    int left = (int)(take - ahead), s = 0;
    while (left > sh.seg_n[s]) left -= sh.seg_n[s++];
    for (int i = 0; i < SL::kIters && left > 0; ++i) {
      const int at = SL::at(s, i);
      float x[SL::N];
      sl.load(at, x);
      int c = 0;
#pragma unroll
      for (int e = 0; e < SL::N; ++e) c += rw.mass.z(x[e]) == zk && sl.base + at + e <= old_idx;
      const int inc = warp_scan(c);
      if (left > inc - c && left <= inc) {
        int nth = left - (inc - c);
#pragma unroll
        for (int e = 0; e < SL::N; ++e)
          if (rw.mass.z(x[e]) == zk && --nth == 0) sh.lo = sl.base + at + e;
      }
      left -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  rw.send(&Mail::tie, sh.lo);
  cluster.sync();
  int idx = -1;
  for (int r = 0; r < (int)cluster.num_blocks(); ++r) idx = max(idx, sh.mail.tie[r]);
  return Cut{zk, idx};
}

// The boundary within the leader's list of n candidates (in vocabulary order), by
// radix selection on the order key; `target` as above.  weight(i): entry i's
// mass in list units, 0 when it has no part in the selection.  Called by all
// threads of the leader.
template <bool MASS, typename W>
__device__ __forceinline__ Cut list_select(Shared& sh, int n, uint64_t target, W weight) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t prefix = 0;
  uint64_t before = 0;  // elements (or mass) ahead of the prefix
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) {
      sh.digit_n[tid] = 0;
      if (MASS) sh.digit_w[tid] = 0;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < n; i += kGivenThreads) {
      const uint32_t k = sh.list.key[i];
      if (shift < 24 && (k >> (shift + 8)) != prefix) continue;
      const int bin = (k >> shift) & 255;
      if (MASS) {
        const uint64_t w = weight(i);
        if (!w) continue;
        atomicAdd(&sh.digit_w[bin], (unsigned long long)w);
      }
      atomicAdd(&sh.digit_n[bin], 1u);
    }
    __syncthreads();
    if (warp == 0) find_digit<MASS>(sh, before, target);
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)sh.bin;
    before = sh.above;
  }
  // the take-th of the elements at the key, in vocabulary order
  if (warp == 0) {
    const uint32_t ties = sh.bin_n;
    int found = kMaxIdx;
    uint32_t seen = 0;
    uint64_t take = 0;
    if (ties > 1) {
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const bool tie = i < n && sh.list.key[i] == prefix && (!MASS || weight(i) > 0);
        const unsigned mask = __ballot_sync(0xffffffffu, tie);
        if (!mask) continue;
        if (take == 0) {
          take = MASS ? (target - before) / weight(i0 + __ffs(mask) - 1) + 1 : target - before;
          if (take >= ties) break;
        }
        const uint32_t nth = seen + __popc(mask & ((1u << lane) - 1)) + 1;
        if (tie && nth == take) found = sh.list.idx[i];
        seen += __popc(mask);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) found = min(found, __shfl_xor_sync(0xffffffffu, found, o));
    }
    if (lane == 0) sh.mail.cut = Cut{key_value(prefix), found};
  }
  __syncthreads();
  return sh.mail.cut;
}

// The threads' sums of seg_n to the elements before each segment; the CTA's
// total is returned to every thread of warp 0.
__device__ __forceinline__ int scan_segments(Shared& sh, int segs) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int s0 = 0; s0 < segs; s0 += 32) {
    const int c = s0 + lane < segs ? sh.seg_n[s0 + lane] : 0;
    const int inc = warp_scan(c) + carry;
    if (s0 + lane < segs) sh.seg_n[s0 + lane] = inc - c;
    carry = __shfl_sync(0xffffffffu, inc, 31);
  }
  return carry;
}

// The elements that `wanted` takes, of every CTA, into the leader's list in
// vocabulary order.  seg_n holds how many each segment has (every warp its own
// segments); `post` sends what else the others need with the same barrier.
// Returns their number in the cluster, or -1 when the list does not hold them.
// The caller's next cluster barrier publishes the list.
template <typename T, bool STAGED, typename F, typename G>
__device__ __forceinline__ int gather(Row<T, STAGED>& rw, F wanted, G post) {
  using SL = Slice<T, STAGED>;
  const SL& sl = rw.sl;
  Shared& sh = rw.sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if (warp == 0) {
    const int c = scan_segments(sh, sl.segs());
    rw.send(&Mail::count, c);
  }
  post();
  cluster.sync();
  int total = 0, base = 0;
  const int rank = cluster.block_rank();
  for (int r = 0; r < (int)cluster.num_blocks(); ++r) {
    if (r == rank) base = total;
    total += sh.mail.count[r];
  }
  if (total > kList) return -1;
  List& list = rw.at(0)->list;
  const int mine = sh.mail.count[rank];
  for (int s = warp; s < sl.segs(); s += kGivenWarps) {
    const int from = sh.seg_n[s], to = s + 1 < sl.segs() ? sh.seg_n[s + 1] : mine;
    if (from == to) continue;
    int off = base + from;
#pragma unroll 1
    for (int i = 0; i < SL::kIters; ++i) {
      const int at = SL::at(s, i);
      float x[SL::N];
      sl.load(at, x);
      unsigned take = 0;
#pragma unroll
      for (int e = 0; e < SL::N; ++e) take |= wanted(x[e], sl.base + at + e) ? 1u << e : 0u;
      if (!__any_sync(0xffffffffu, take)) continue;
      const int c = __popc(take);
      const int inc = warp_scan(c);
      int p = off + inc - c;
#pragma unroll
      for (int e = 0; e < SL::N; ++e)
        if ((take >> e) & 1) {
          list.key[p] = ord_key(rw.mass.z(x[e]));
          list.idx[p] = sl.base + at + e;
          ++p;
        }
      off += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  return total;
}

// Elements kept by a cut in the linear bins lo .. hi.
template <typename T, bool STAGED>
struct InBins {
  const Row<T, STAGED>& rw;
  Cut cut;
  int lo, hi;
  __device__ __forceinline__ bool operator()(float x, int j) const {
    const float z = rw.mass.z(x);
    const int bin = bin_of(rw.bins_below(z));
    return cut.keeps(z, j) && bin >= lo && bin <= hi;
  }
};

constexpr int kListDrop = 2;  // list masses: units of 2^(E - kElemBits + 2), 2048 below 2^62

// The boundary of the elements kept by `cut` by one linear histogram below the
// maximum, which brackets it, and a list of the elements in the bracket.
//   MASS: target is the top-p share `p`; on success the CTAs' seg_w hold the
//   masses of the kept elements (element units) and *row_mass the mass of all
//   elements kept by `cut`.
//   else: the first `top_k` are kept.
// Returns false (the same in every CTA) when the bracket holds too many, or, by
// mass, turns out not to hold the boundary.
template <typename T, bool STAGED, bool MASS>
__device__ __noinline__ bool band_select(const Row<T, STAGED>& row_in, Cut* cut_io, float p,
                                         int top_k, uint64_t* row_mass) {
  Row<T, STAGED> rw = row_in;  // in registers
  using SL = Slice<T, STAGED>;
  const SL& sl = rw.sl;
  Shared& sh = rw.sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const Cut cut = *cut_io;
  constexpr int kPer = kBins / kGivenThreads;
#pragma unroll
  for (int q = 0; q < kPer; ++q) sh.hist.own[tid + q * kGivenThreads] = 0;
  if (tid == 0) {
    sh.lo = kBins;
    sh.hi = -1;
  }
  __syncthreads();
  // by mass: each element adds its mass relative to its bin's upper edge in
  // units of 1/4095, so a bin's mass is known to within 1.3e-4 of itself
  for (int s = warp; s < sl.segs(); s += kGivenWarps) {
#pragma unroll 1
    for (int i = 0; i < SL::kIters; ++i) {
      const int at = SL::at(s, i);
      float x[SL::N];
      sl.load(at, x);
#pragma unroll
      for (int e = 0; e < SL::N; ++e) {
        const float z = rw.mass.z(x[e]);
        const float t = rw.bins_below(z);
        const int bin = bin_of(t);
        uint32_t add = 1;
        if (MASS) {
          const float f = t - (float)bin;
          add = (uint32_t)__fmaf_rn(f, __fmaf_rn(f, 0.4999f, -63.984f), 4095.5f);
        }
        if (cut.keeps(z, sl.base + at + e) && !(MASS && bin == kBins - 1))
          atomicAdd(&sh.hist.own[bin], add);
      }
    }
  }
  // the cluster's histogram: CTA r sums a share of the bins and sends it to all
  cluster.sync();
  const int share = kBins / C;
  for (int q = tid; q < share; q += kGivenThreads) {
    const int bin = rank * share + q;
    uint32_t c = 0;
    for (int r = 0; r < C; ++r) c += rw.at(r)->hist.own[bin];
    for (int r = 0; r < C; ++r) rw.at(r)->hist.sum[bin] = c;
  }
  cluster.sync();
  uint32_t cn[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) cn[q] = sh.hist.sum[tid * kPer + q];
  uint64_t above_n = 0;  // elements above the bracket (by count)
  if (MASS) {
    float cf[kPer], tf = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      cf[q] = (float)cn[q] * ex2_approx((float)(tid * kPer + q) * (-kLog2e / kBinsPerNat));
      tf += cf[q];
    }
    float inc = warp_scan(tf);
    if (lane == 31) sh.red_f[warp] = inc;
    __syncthreads();
    float a = inc - tf, all = 0.f;
    for (int i = 0; i < kGivenWarps; ++i) {
      if (i < warp) a += sh.red_f[i];
      all += sh.red_f[i];
    }
    constexpr float kSlack = 1.f / 6144;  // of the bins' masses and their fp32 sums
    const float want = p * all;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (cn[q] > 0) {
        // bins that end before the target are kept whole, those that begin
        // after it not at all
        if (a + cf[q] >= want * (1.f - kSlack)) atomicMin(&sh.lo, tid * kPer + q);
        if (a <= want * (1.f + kSlack)) atomicMax(&sh.hi, tid * kPer + q);
      }
      a += cf[q];
    }
  } else {
    uint64_t tn = 0, unused;
#pragma unroll
    for (int q = 0; q < kPer; ++q) tn += cn[q];
    uint64_t a = block_scan(sh, tn, &unused);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (a < (uint64_t)top_k && a + cn[q] >= (uint64_t)top_k) {
        sh.lo = sh.hi = tid * kPer + q;
        sh.above = a;
      }
      a += cn[q];
    }
  }
  __syncthreads();
  const int lo = sh.lo, hi = sh.hi;
  if (!MASS) above_n = sh.above;
  if (lo > hi) return false;  // (a histogram without mass)

  uint64_t w_above = 0, w_all = 0;
  for (int s = warp; s < sl.segs(); s += kGivenWarps) {
    uint64_t above = 0, rest = 0;
    int c = 0;
#pragma unroll 1
    for (int i = 0; i < SL::kIters; ++i) {
      const int at = SL::at(s, i);
      float x[SL::N];
      sl.load(at, x);
#pragma unroll
      for (int e = 0; e < SL::N; ++e) {
        const float z = rw.mass.z(x[e]);
        const bool in = cut.keeps(z, sl.base + at + e);
        const int bin = bin_of(rw.bins_below(z));
        c += in && bin >= lo && bin <= hi;
        if (MASS) {
          const uint64_t w = in ? rw.mass.of(z) : 0;
          above += bin < lo ? w : 0;
          rest += w;
        }
      }
    }
    c = warp_sum_i(c);
    if (MASS) {
      above = warp_sum_u64(above);
      rest = warp_sum_u64(rest);
    }
    if (lane == 0) {
      sh.seg_n[s] = c;
      if (MASS) {
        sh.seg_w[s] = above;
        w_above += rw.coarse(above);
        w_all += rw.coarse(rest);
      }
    }
  }
  if (MASS && lane == 0) {
    sh.red_w[warp] = w_above;
    sh.red_n[warp] = w_all;
  }
  const int n = gather(rw, InBins<T, STAGED>{rw, cut, lo, hi}, [&]() {
    if (MASS && warp == 0) {
      w_above = warp_sum_u64(lane < kGivenWarps ? sh.red_w[lane] : 0);
      w_all = warp_sum_u64(lane < kGivenWarps ? sh.red_n[lane] : 0);
      rw.send(&Mail::mass, w_above);
      rw.send(&Mail::all, w_all);
    }
  });
  if (MASS) {
    w_above = w_all = 0;
    for (int r = 0; r < C; ++r) {
      w_above += sh.mail.mass[r];
      w_all += sh.mail.all[r];
    }
    *row_mass = w_all;
  }
  cluster.sync();
  if (n <= 0) return false;
  if (rank == 0) {
    bool ok = true;
    Cut found{0.f, kMaxIdx};
    if (MASS) {
      auto weight = [&](int i) { return (rw.mass.of(key_value(sh.list.key[i])) + 2) >> kListDrop; };
      uint64_t mine = 0, band;
      for (int i = tid; i < n; i += kGivenThreads) mine += weight(i);
      block_scan(sh, mine, &band);
      const uint64_t target = part_of(w_all, p);
      // the boundary lies in the bracket: the mass above it is within the
      // target, that at its end is not
      ok = w_above <= target && (target - w_above) < (1ull << (62 - rw.drop));
      const uint64_t left = ok ? (target - w_above) << (rw.drop - kListDrop) : 0;
      ok = ok && left < band;
      if (ok) found = list_select<true>(sh, n, left, weight);
      if (ok)
        for (int i = tid; i < n; i += kGivenThreads) {
          const int j = sh.list.idx[i];
          const float z = key_value(sh.list.key[i]);
          if (found.keeps(z, j)) {
            const int r = j / rw.slice;
            atomicAdd((unsigned long long*)&rw.at(r)->seg_w[(j - r * rw.slice) / kSeg],
                      (unsigned long long)rw.mass.of(z));
          }
        }
    } else {
      found = list_select<false>(sh, n, (uint64_t)top_k - above_n, [](int) { return 1ull; });
    }
    if (tid < C) {
      rw.at(tid)->mail.cut = found;
      rw.at(tid)->mail.ok = ok;
    }
  }
  cluster.sync();
  if (sh.mail.ok) *cut_io = sh.mail.cut;
  return sh.mail.ok;
}

// Masses of the kept elements by segment, into seg_w (element units).
template <typename T, bool STAGED>
__device__ __noinline__ void kept_mass(const Row<T, STAGED>& row_in, const Cut cut) {
  Row<T, STAGED> rw = row_in;  // in registers
  using SL = Slice<T, STAGED>;
  const SL& sl = rw.sl;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int s = warp; s < sl.segs(); s += kGivenWarps) {
    uint64_t w = 0;
#pragma unroll 1
    for (int i = 0; i < SL::kIters; ++i) {
      const int at = SL::at(s, i);
      float x[SL::N];
      sl.load(at, x);
#pragma unroll
      for (int e = 0; e < SL::N; ++e) {
        const float z = rw.mass.z(x[e]);
        const uint64_t v = rw.mass.of(z);
        w += cut.keeps(z, sl.base + at + e) ? v : 0;
      }
    }
    w = warp_sum_u64(w);
    if (lane == 0) rw.sh.seg_w[s] = w;
  }
}

// seg_w to inclusive sums in row units; returns the cluster's total, the mass of
// the CTAs before this one and this CTA's.
template <typename T, bool STAGED>
__device__ uint64_t sum_segments(Row<T, STAGED>& rw, uint64_t* before, uint64_t* own) {
  Shared& sh = rw.sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, segs = rw.sl.segs();
  __syncthreads();
  if (warp == 0) {
    uint64_t carry = 0;
    for (int s0 = 0; s0 < segs; s0 += 32) {
      const uint64_t w =
          warp_scan(s0 + lane < segs ? rw.coarse(sh.seg_w[s0 + lane]) : (uint64_t)0) + carry;
      if (s0 + lane < segs) sh.seg_w[s0 + lane] = w;
      carry = __shfl_sync(0xffffffffu, w, 31);
    }
    rw.send(&Mail::kept, carry);
  }
  cluster.sync();
  uint64_t total = 0;
  const int rank = cluster.block_rank();
  for (int r = 0; r < (int)cluster.num_blocks(); ++r) {
    if (r == rank) *before = total;
    total += sh.mail.kept[r];
  }
  *own = sh.mail.kept[rank];
  return total;
}

// The first kept element of this CTA whose inclusive mass (from the CTA's start)
// exceeds t (row units, below the CTA's mass); one warp.
template <typename T, bool STAGED>
__device__ int find_draw(const Row<T, STAGED>& rw, const Cut& cut, uint64_t t, float* z_out) {
  using SL = Slice<T, STAGED>;
  const SL& sl = rw.sl;
  const int lane = threadIdx.x & 31;
  int s = 0;
  for (int s0 = 0; s0 < sl.segs(); s0 += 32) {
    const bool past = s0 + lane < sl.segs() && rw.sh.seg_w[s0 + lane] <= t;
    s += __popc(__ballot_sync(0xffffffffu, past));
  }
  if (s > 0) t -= rw.sh.seg_w[s - 1];
  t <<= rw.drop;  // element units
  int idx = -1;
  float zz = 0.f;
  for (int i = 0; i < SL::kIters; ++i) {
    const int at = SL::at(s, i);
    float x[SL::N];
    sl.load(at, x);
    uint64_t w[SL::N], sum = 0;
#pragma unroll
    for (int e = 0; e < SL::N; ++e) {
      const float z = rw.mass.z(x[e]);
      w[e] = cut.keeps(z, sl.base + at + e) ? rw.mass.of(z) : 0;
      sum += w[e];
    }
    const uint64_t inc = warp_scan(sum);
    uint64_t run = inc - sum;
    // the segment's sum was rounded to row units: a t within that of its end
    // takes the last element that has mass
    int here = -1, last = -1;
    float z_here = 0.f, z_last = 0.f;
#pragma unroll
    for (int e = 0; e < SL::N; ++e) {
      run += w[e];
      if (w[e] > 0) {
        last = sl.base + at + e;
        z_last = rw.mass.z(x[e]);
        if (here < 0 && run > t) {
          here = last;
          z_here = z_last;
        }
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, here >= 0);
    if (hit) {
      const int owner = __ffs(hit) - 1;
      *z_out = __shfl_sync(0xffffffffu, z_here, owner);
      return __shfl_sync(0xffffffffu, here, owner);
    }
    const unsigned any = __ballot_sync(0xffffffffu, last >= 0);
    if (any) {
      const int owner = 31 - __clz(any);
      zz = __shfl_sync(0xffffffffu, z_last, owner);
      idx = __shfl_sync(0xffffffffu, last, owner);
    }
    t -= __shfl_sync(0xffffffffu, inc, 31);
  }
  *z_out = zz;
  return idx;
}

// Threads whose maximum counts as one group, for a row of C CTAs: so many groups
// that at least twice top_k remain.  0: the row has too few threads.
__device__ __forceinline__ int group_threads(int C, int top_k) {
  if (top_k < 2 || top_k > kListTopK || 2 * top_k > C * kGivenThreads) return 0;
  int g = 1;
  while (g < 32 && C * kGivenThreads / (2 * g) >= 2 * top_k) g *= 2;
  return g;  // at most 2 * kListTopK groups, both powers of two
}

// A row with 1 < top_k <= kListTopK: the maxima of groups of elements (in
// hist.group_max) give a value that at least top_k elements reach; those elements
// go to the leader's list, where min-p, top-k and top-p are settled and the draws
// made.  Adds ln sum exp on the way.  Returns false (in every CTA) when the list
// does not hold them.
template <typename T, bool STAGED>
__device__ __noinline__ bool draw_from_list(const Row<T, STAGED>& row_in, const GivenArgs& a,
                                            const RowParams& P, const Cut minp, int groups,
                                            int row, float* ln_s_out) {
  Row<T, STAGED> rw = row_in;  // in registers
  using SL = Slice<T, STAGED>;
  const SL& sl = rw.sl;
  Shared& sh = rw.sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kPer = kBins / kGivenThreads;
#pragma unroll
  for (int q = 0; q < kPer; ++q) sh.hist.own[tid + q * kGivenThreads] = 0;
  if (tid == 0) sh.hi = kBins - 1;
  __syncthreads();
  for (int i = tid; i < groups; i += kGivenThreads) {
    const float x = sh.hist.group_max[i];
    if (x > -INFINITY) atomicAdd(&sh.hist.own[bin_of(rw.bins_below(rw.mass.z(x)))], 1u);
  }
  __syncthreads();
  {
    uint32_t cn[kPer];
    uint64_t tn = 0, unused;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      cn[q] = sh.hist.own[tid * kPer + q];
      tn += cn[q];
    }
    uint64_t b = block_scan(sh, tn, &unused);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (b < (uint64_t)P.top_k && b + cn[q] >= (uint64_t)P.top_k) sh.hi = tid * kPer + q;
      b += cn[q];
    }
  }
  __syncthreads();
  // (fewer than top_k groups with a finite element: every finite element)
  const float edge = sh.hi == kBins - 1 ? INFINITY : (float)(sh.hi + 1);
  float expsum = 0.f;
  for (int s = warp; s < sl.segs(); s += kGivenWarps) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < SL::kIters; ++i) {
      float x[SL::N];
      sl.load(SL::at(s, i), x);
#pragma unroll
      for (int e = 0; e < SL::N; ++e) {
        const float t = rw.bins_below(rw.mass.z(x[e]));
        c += t < edge;
        expsum += ex2_approx(__fmul_rn(t, -kLog2e / kBinsPerNat));
      }
    }
    c = warp_sum_i(c);
    if (lane == 0) sh.seg_n[s] = c;
  }
  expsum = block_sum(sh, expsum);
  const int n = gather(rw, [&](float x, int) { return rw.bins_below(rw.mass.z(x)) < edge; },
                       [&]() { rw.send(&Mail::expsum, expsum); });
  expsum = 0.f;
  for (int r = 0; r < (int)cluster.num_blocks(); ++r) expsum += sh.mail.expsum[r];
  const float ln_s = logf(expsum);
  *ln_s_out = ln_s;
  cluster.sync();
  if (n < 0) return false;
  if (cluster.block_rank() != 0) return true;

  const List& list = sh.list;
  Cut cut = minp;
  int kept = 0;
  for (int i = tid; i < n; i += kGivenThreads) kept += key_value(list.key[i]) >= cut.z;
  kept = block_sum(sh, kept);
  // (elements that min-p leaves out come after the others in the order)
  if (kept > P.top_k)
    cut = list_select<false>(sh, n, (uint64_t)P.top_k, [](int) { return 1ull; });
  auto weight = [&](int i) -> uint64_t {
    if (i >= n) return 0;
    const float z = key_value(list.key[i]);
    return cut.keeps(z, list.idx[i]) ? (rw.mass.of(z) + 2) >> kListDrop : 0;
  };
  // each thread holds a few neighbours of the list
  auto own = [&]() {
    uint64_t sum = 0;
#pragma unroll
    for (int q = 0; q < kListPerThread; ++q) sum += weight(tid * kListPerThread + q);
    return sum;
  };
  uint64_t total, mine = own();
  uint64_t ahead = block_scan(sh, mine, &total);
  if (P.flags & kRowTopP) {
    const Cut next = list_select<true>(sh, n, part_of(total, P.top_p), weight);
    cut = next;
    mine = own();
    ahead = block_scan(sh, mine, &total);
  }
  sh.run[tid] = ahead + mine;
  __syncthreads();
  for (int d = tid; d < a.draws; d += kGivenThreads) {
    const int64_t o = (int64_t)row * a.draws + d;
    const uint64_t t = part_of(total, a.uniforms[o]);
    int lo = 0, hi = kGivenThreads - 1;  // the first thread whose inclusive mass exceeds t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sh.run[mid] > t) hi = mid;
      else lo = mid + 1;
    }
    uint64_t run = lo > 0 ? sh.run[lo - 1] : 0;
    int i = lo * kListPerThread;
    for (run += weight(i); run <= t; run += weight(i)) ++i;
    a.out_tokens[o] = list.idx[i];
    if (a.out_logprobs)
      a.out_logprobs[o] = __fsub_rn(__fsub_rn(key_value(list.key[i]), rw.m), ln_s);
  }
  return true;
}

template <typename T, bool STAGED>
__global__ void __launch_bounds__(kGivenThreads, 2) given_kernel(GivenArgs a) {
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
      if (c * chunk < n_bulk && !mbar_wait_bounded(&sh.bars[c], 0))
        atomicOr(a.err_word, kErrTimeout);
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
  // the maximum to every CTA, and for a top-k row the maxima of groups of threads
  const bool greedy = P.flags & kRowGreedy;
  const bool topk = !greedy && P.top_k > 1 && P.top_k < a.V;
  const int group = topk ? group_threads(C, P.top_k) : 0;
  float gmax = mx;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o < group) gmax = max_nan(gmax, __shfl_xor_sync(0xffffffffu, gmax, o));
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (lane == 0) sh.red_f[warp] = mx;
  cluster.sync();  // every CTA of the cluster runs before its memory is written
  if (group && (tid & (group - 1)) == 0)
    for (int r = 0; r < C; ++r)
      cluster.map_shared_rank(&sh, r)->hist.group_max[rank * (kGivenThreads / group) + tid / group] =
          gmax;
  if (tid < C) {
    mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kGivenWarps; ++i) mx = max_nan(mx, sh.red_f[i]);
    cluster.map_shared_rank(&sh, tid)->mail.max[rank] = mx;
  }
  cluster.sync();
  mx = -INFINITY;
  for (int r = 0; r < C; ++r) mx = max_nan(mx, sh.mail.max[r]);
  const float m = __fmul_rn(mx, P.inv_t);
  const int status = isnan(mx) || m == INFINITY ? kRowNonfinite : m == -INFINITY ? kRowEmpty : kRowOk;
  if (rank == 0 && tid == 0) a.row_status[row] = status;
  int32_t* out_tok = a.out_tokens + (int64_t)row * a.draws;
  float* out_lp = a.out_logprobs ? a.out_logprobs + (int64_t)row * a.draws : nullptr;
  if (status != kRowOk) {
    for (int d = rank * kGivenThreads + tid; d < a.draws; d += C * kGivenThreads) {
      out_tok[d] = -1;
      if (out_lp) out_lp[d] = NAN;
    }
    return;
  }
  const Mass mass(P.inv_t, m, sh.table);
  Row<T, STAGED> rw(sl, sh, mass, m, a.slice, a.drop);

  Cut cut{-3.402823466e38f, kMaxIdx};
  if ((P.flags & kRowMinP) && !(P.flags & kRowGreedy)) {
    // the smallest z with z - m >= ln(min_p), both sides in double
    float zt = __double2float_rn((double)m + P.log_min_p);
    if ((double)zt - (double)m < P.log_min_p) {
      zt = nextafterf(zt, INFINITY);
    } else {
      const float below = nextafterf(zt, -INFINITY);
      if ((double)below - (double)m >= P.log_min_p) zt = below;
    }
    cut.z = fmaxf(cut.z, zt);
  }
  float ln_s = 0.f;
  bool have_ln_s = false;
  if (group) {
    if (draw_from_list(rw, a, P, cut, C * kGivenThreads / group, row, &ln_s)) return;
    have_ln_s = true;
  }

  // ln sum exp(z - m) where the masses will not give it; a greedy row's lowest
  // index at the maximum
  const bool all_mass = !greedy && !topk && !(P.flags & kRowMinP);
  if (greedy || (out_lp && !have_ln_s && !all_mass)) {
    float expsum = 0.f;
    int first = kMaxIdx;
    for (int s = warp; s < sl.segs(); s += kGivenWarps) {
#pragma unroll
      for (int i = 0; i < SL::kIters; ++i) {
        const int at = SL::at(s, i);
        float x[SL::N];
        sl.load(at, x);
#pragma unroll
        for (int e = 0; e < SL::N; ++e) {
          expsum += ex2_approx(__fmul_rn(__fsub_rn(rw.mass.z(x[e]), m), kLog2e));
          if (greedy && x[e] == mx) first = min(first, sl.base + at + e);
        }
      }
    }
    expsum = block_sum(sh, expsum);
    rw.send(&Mail::expsum, expsum);
    if (greedy) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
      if (lane == 0) sh.red_i[warp] = first;
      __syncthreads();
      if (tid < C)
        for (int i = 0; i < kGivenWarps; ++i) first = min(first, sh.red_i[i]);
      rw.send(&Mail::index, first);
    }
    cluster.sync();
    expsum = 0.f;
    first = kMaxIdx;
    for (int r = 0; r < C; ++r) {
      expsum += sh.mail.expsum[r];
      if (greedy) first = min(first, sh.mail.index[r]);
    }
    ln_s = logf(expsum);
    if (greedy) {
      for (int d = rank * kGivenThreads + tid; d < a.draws; d += C * kGivenThreads) {
        out_tok[d] = first;
        if (out_lp) out_lp[d] = -ln_s;
      }
      return;
    }
  }

  // the kept set
  if (topk) {
    // (an element count decides whether top-k cuts anything)
    int c = 0;
    for (int s = warp; s < sl.segs(); s += kGivenWarps) {
#pragma unroll 1
      for (int i = 0; i < SL::kIters; ++i) {
        float x[SL::N];
        sl.load(SL::at(s, i), x);
#pragma unroll
        for (int e = 0; e < SL::N; ++e) c += rw.mass.z(x[e]) >= cut.z;
      }
    }
    rw.send(&Mail::total, block_sum(sh, c));
    cluster.sync();
    int n = 0;
    for (int r = 0; r < C; ++r) n += sh.mail.total[r];
    if (n > P.top_k && !band_select<T, STAGED, false>(rw, &cut, 0.f, P.top_k, nullptr))
      cut = radix_select<T, STAGED, false>(rw, cut, (uint64_t)P.top_k);
  }
  uint64_t before, mine, W, all;
  if (P.flags & kRowTopP) {
    const Cut from = cut;
    if (!band_select<T, STAGED, true>(rw, &cut, P.top_p, 0, &all)) {
      kept_mass(rw, from);
      all = sum_segments(rw, &before, &mine);
      cut = radix_select<T, STAGED, true>(rw, from, part_of(all, P.top_p));
      kept_mass(rw, cut);
    }
    W = sum_segments(rw, &before, &mine);
  } else {
    kept_mass(rw, cut);
    W = all = sum_segments(rw, &before, &mine);
  }
  if (all_mass) ln_s = rw.mass.ln_sum(all, kElemBits - a.drop, m);

  // the draws: each by a warp of the CTA that holds its mass
  for (int d = warp; d < a.draws; d += kGivenWarps) {
    const uint64_t t = part_of(W, a.uniforms[(int64_t)row * a.draws + d]);
    if (t < before || t - before >= mine) continue;
    float z;
    const int j = find_draw(rw, cut, t - before, &z);
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
  while (cluster < kMaxCtas && ((int64_t)slice_of(cluster) * es > 80 * 1024 ||
                                slice_of(cluster) > kSeg * kMaxSegs ||
                                ((int64_t)a.B * cluster * 2 <= 2 * num_sms &&
                                 slice_of(cluster) > 4096)))
    cluster *= 2;
  a.slice = slice_of(cluster);
  // sums of V masses stay below 2^62
  int bits = 0;
  while ((1ll << bits) < a.V) ++bits;
  a.drop = max(kListDrop, bits + kElemBits - 62);
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
