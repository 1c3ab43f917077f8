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
// order, and a mass is within 1.1e-9 (rms 2.8e-10) of exp() in relative terms.  A
// prefix of N such errors moves a boundary by about 2.8e-10 / sqrt(N) of W (N the
// distinct values among bf16 logits, a hundred and more), which puts the chance of
// a draw differing from the exact one below 1e-5 for a flat row of 151,936.
//
// Two launches.  stream_kernel reads the logits once: a warp takes 1024 of them
// into registers and leaves their maximum, the maxima of their 64-element groups
// and their sum of masses (or of exponentials), relative to their own maximum,
// so that nothing waits for the row's.  finish_kernel settles each row from these
// and reads again only the segments and groups that can matter: one segment for
// an unfiltered or greedy row's token, the groups that reach the top_k-th group
// maximum, the whole row (from L2) only for top-p over everything.
// What bounds them: stream_kernel HBM where few rows need sums of masses, else
// the 24 instructions of a mass (1024 fp32 rows of 248,320, 1.02 GB: 185 us when
// no row does, 286 us when all do); finish_kernel the chain of block-wide steps
// of a row, and for top-p rows their two passes over the elements (256 bf16 rows
// of 151,936: 18 us greedy, 27 unfiltered, 37 top-k 20, 143 top-p 0.9).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "vt_device.cuh"
#include "vt_kernels.h"
#include "vt_sampler.h"

namespace cg = cooperative_groups;

namespace vt {
namespace {

constexpr int kStreamThreads = 256;
constexpr int kStreamCtas = 3;      // an SM (with four, 213 us instead of 187)
constexpr int kThreadsF = 512;      // of finish_kernel
constexpr int kWarpsF = kThreadsF / 32;
constexpr int kSeg = kGivenSeg;     // elements a warp takes at a time, in vocabulary order
constexpr int kGroup = kGivenGroup; // elements that share a group maximum
constexpr int kGroupsPerSeg = kSeg / kGroup;
constexpr int kMaxSegs = 1024;      // of a row: V <= 2^20
constexpr int kMaxCtas = 16;        // CTAs that finish a row
constexpr int kBins = 4096;
constexpr float kBinsPerLogit = 128.f;  // linear bins: 32 logits below the maximum, then one for all
constexpr int kList = 2048;         // candidates a row's leader CTA holds
constexpr int kListTopK = 1024;     // largest top-k taken from group maxima
constexpr int kListPerThread = kList / kThreadsF;
constexpr int kMaxIdx = 0x7fffffff;
constexpr float kNarrow = 5000.f;   // maxima beyond: masses relative to the maximum itself
constexpr float kUsable = 4900.f;   // maxima beyond: the segments' sums are not used

constexpr int kTable = 512, kTableLog = 9;
constexpr int kElemBits = 53;   // masses of single elements: units of 2^-53 of 2^E
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: x + kMagic holds rint(x) in its low bits
constexpr float kMagic512 = 24576.f;  // 1.5 * 2^14: x + kMagic512 holds rint(512 x)
constexpr uint32_t kMagicBits = 0x4b400000u, kMagic512Bits = 0x46c00000u;

// 2^(i/512) in units of 2^-30, from powers of 2^(1/512): as an integer less
// kMagicBits, and as a float.
struct MassTable {
  uint2 v[kTable];
  constexpr MassTable() : v() {
    double x = 1073741824.0;
    for (int i = 0; i < kTable; ++i) {
      v[i].x = (uint32_t)(x + 0.5) - kMagicBits;
      v[i].y = float_bits(x);
      x *= 1.0013547198921082;
    }
  }
  // the bits of the float next to x, 2^30 <= x < 2^31
  static constexpr uint32_t float_bits(double x) {
    return ((127u + 30u) << 23) + (uint32_t)((x - 1073741824.0) / 128.0 + 0.5);
  }
};
// (not in constant memory: lanes that read other entries would take turns)
__device__ const MassTable d_mass_table = MassTable();

// x >> n, 0 from 32 on.
__device__ __forceinline__ uint32_t shr(uint32_t x, int n) {
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(n));
  return r;
}

// Masses as integers: exp(z) = 2^(z log2(e)) relative to 2^E, the power of two
// next above the maximum, so that no subtraction of the maximum rounds.
//   k = the multiple of 1/512 next to z log2(e), r = z log2(e) - k in [-1/1024,
//   1/1024] by two FMAs (exact to 2^-34): the mass is 2^floor(k) *
//   table[512 frac(k)] * 2^r, with 2^r - 1 as a quadratic (within 2^-34), the
//   mantissa an integer in units of 2^-30.
// Its error: half a unit of 2^-30 by the table's rounding and half a one by the sum's
// (4.7e-10 each where the mantissa is 1), 5.2e-11 by the quadratic, 4e-11 by r.
// 24 instructions: roundings to integers go by the two magic numbers, not by
// conversions (an eighth of the rate), the mantissa by an FMA, not by an integer
// product.  For a maximum beyond 5000 the reduction would run out of bits;
// there z - m is exact wherever the mass is not 0 (z within a factor 2 of m), so
// the row's values are shifted by c = m (else c = 0).
struct Mass {
  float inv_t, c, floor_z;
  uint32_t e_bits;  // kMagic512Bits + kTable * E + kTable - 1
  const uint2* table;

  __device__ __forceinline__ Mass(float inv_t_, float m, const uint2* table_) {
    inv_t = inv_t_;
    table = table_;
    c = fabsf(m) < kNarrow ? 0.f : m;
    const int E = (int)floorf(__fmul_rn(m - c, kLog2e)) + 1;
    e_bits = kMagic512Bits + (uint32_t)(E * kTable + kTable - 1);
    floor_z = (float)(E - 56) * kLn2;  // shifted out whole: -inf and far below have mass 0
  }
  __device__ __forceinline__ int E() const {
    return ((int)(e_bits - kMagic512Bits) - (kTable - 1)) >> kTableLog;
  }
  __device__ __forceinline__ float z(float x) const { return __fmul_rn(x, inv_t); }
  // mass of the tempered value z, truncated to units of 2^(E - kElemBits), added to acc
  __device__ __forceinline__ uint64_t add(uint64_t acc, float z) const {
    z = fmaxf(__fsub_rn(z, c), floor_z);
    const float kb = __fmaf_rn(z, kLog2e, kMagic512);
    float r = __fmaf_rn(z, kLog2e, -__fsub_rn(kb, kMagic512));
    r = __fmaf_rn(z, 1.92596303e-8f, r);  // log2(e) - fl(log2(e))
    const float q = __fmul_rn(r, __fmaf_rn(r, 0.240226507f, 0.693147181f));
    const uint32_t k = __float_as_uint(kb);
    const uint2 t = *reinterpret_cast<const uint2*>(reinterpret_cast<const char*>(table) +
                                                    ((k << 3) & ((kTable - 1) << 3)));
    const uint32_t mant = t.x + __float_as_uint(__fmaf_rn(q, __uint_as_float(t.y), kMagic));
    // mant 2^(kElemBits - 30 - n), n = E - floor(k) >= 0
    const int n = (int)(e_bits - k) >> kTableLog;
    constexpr int kUp = kElemBits - 30;
    const uint32_t lo = shr(mant, max(n - kUp, 0));
    const uint32_t up = max(shr(1u << kUp, n), 1u);
    return acc + (uint64_t)lo * up;
  }
  __device__ __forceinline__ uint64_t of(float z) const { return add(0, z); }
  // ln of a sum of masses in units of 2^(E - bits), relative to the maximum m
  __device__ __forceinline__ float ln_sum(uint64_t w, int bits, float m) const {
    const float e = (float)E();
    const float lw = logf(__ull2float_rn(w) * exp2f((float)-bits));
    // E ln 2 - (m - c) in one rounding, ln 2 in two parts
    return lw + (__fmaf_rn(e, 0.693147182464599609375f, -__fsub_rn(m, c)) +
                 e * -1.904654299957e-9f);
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

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float max(const uint4& v) {
    const uint32_t u = max2(max2(v.x, v.y), max2(v.z, v.w));
    return max_nan(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
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
  static __device__ __forceinline__ float max(const uint4& v) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                   max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
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

// One row's logits in global memory.
template <typename T>
struct RowData {
  static constexpr int N = Vec<T>::N;           // elements of a 16-byte load
  static constexpr int kIters = kSeg / (32 * N);
  const T* data;
  int V;
  bool vec;  // 16-byte loads
  // position of the first of a lane's N elements in iteration i of segment s
  static __device__ __forceinline__ int at(int s, int i) {
    return s * kSeg + (i * 32 + (int)(threadIdx.x & 31)) * N;
  }
  __device__ __forceinline__ uint4 raw(int p) const {
    if (vec && p + N <= V) return __ldg(reinterpret_cast<const uint4*>(data + p));
    alignas(16) T x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = p + i < V ? data[p + i] : static_cast<T>(-INFINITY);
    return *reinterpret_cast<const uint4*>(x);
  }
  // elements p .. p + N - 1; -inf past the row's end
  __device__ __forceinline__ void load(int p, float (&x)[N]) const { Vec<T>::unpack(raw(p), x); }
};

// f(x, p) on the N elements from p on of every lane, over segment s in order.
// Four loads are in flight; the body is there once, whatever the element type,
// because the first pass of a row through long unrolled code is bound by
// instruction fetches.
template <typename T, typename F>
__device__ __forceinline__ void each_vector(const RowData<T>& rd, int s, F f) {
  using RD = RowData<T>;
#pragma unroll 1
  for (int h = 0; h < RD::kIters; h += 4) {
    uint4 v0 = rd.raw(RD::at(s, h)), v1 = rd.raw(RD::at(s, h + 1)), v2 = rd.raw(RD::at(s, h + 2)),
          v3 = rd.raw(RD::at(s, h + 3));
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      float x[RD::N];
      Vec<T>::unpack(v0, x);
      v0 = v1;
      v1 = v2;
      v2 = v3;
      f(x, RD::at(s, h + i));
    }
  }
}

// Exponentials for the log-probs are 2^(z log2(e) - lse_base(max)): one FMA, with
// the values of a far maximum shifted by it first, as in struct Mass.
__device__ __forceinline__ float lse_shift(float zm) { return fabsf(zm) < kNarrow ? 0.f : zm; }
__device__ __forceinline__ float lse_base(float zm) {
  return __fmul_rn(zm - lse_shift(zm), kLog2e);
}

// Whether a row's segments are summed as masses (else as exponentials for the
// log-probs): rows whose kept mass, or top-p total, is that of every element.
__device__ __forceinline__ bool sums_masses(const RowParams& P, int V) {
  return !(P.flags & (kRowGreedy | kRowMinP)) && !(P.top_k > 1 && P.top_k < V);
}

// One warp to a segment of 1024 logits, in registers (bf16: four 16-byte loads a
// lane, fp32 eight).  The next segment is on its way into the warp's own buffer of
// shared memory, by one bulk copy, while this one is worked on (without that the
// loads pause for the arithmetic: 1024 fp32 rows 210 us); segments that a bulk copy
// cannot take (unaligned rows, a row's ragged end) are loaded directly, and so are
// the rest of a warp's, once a wait for a copy has run out.  What bounds it: HBM.
template <typename T>
__global__ void __launch_bounds__(kStreamThreads, kStreamCtas) stream_kernel(GivenArgs a) {
  using RD = RowData<T>;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ uint2 table[kTable];
  __shared__ uint64_t bars[kStreamThreads / 32];
  for (int i = threadIdx.x; i < kTable; i += kStreamThreads) table[i] = d_mass_table.v[i];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint4* buf = reinterpret_cast<const uint4*>(dyn) + warp * (kSeg * sizeof(T) / 16);
  if (lane == 0) mbar_init(&bars[warp], 1);
  fence_mbar_init();
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");
  const uint32_t items = (uint32_t)a.B * a.segs, step = gridDim.x * (kStreamThreads / 32);
  // whether segment `it` comes by a bulk copy, and the copy
  bool copies = a.aligned != 0, late = false;
  auto by_copy = [&](uint32_t it) {
    return copies && it < items && (int)(it % a.segs + 1) * kSeg <= a.V;
  };
  auto fetch = [&](uint32_t it) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[warp], kSeg * sizeof(T));
      bulk_copy_g2s(const_cast<uint4*>(buf),
                    static_cast<const T*>(a.logits) + (it / a.segs) * a.ld +
                        (int64_t)(it % a.segs) * kSeg,
                    kSeg * sizeof(T), &bars[warp]);
    }
  };
  uint32_t it = blockIdx.x * (kStreamThreads / 32) + warp, phase = 0;
  if (by_copy(it)) fetch(it);
  for (; it < items; it += step) {
    const int row = (int)(it / a.segs), seg = (int)(it % a.segs);
    uint4 v[RD::kIters];
    bool here = by_copy(it);
    if (here) {
      here = __all_sync(0xffffffffu,
                        a.wait_cycles > 0 && mbar_wait_clocked(&bars[warp], phase, a.wait_cycles));
      if (!here) {  // this copy is the one in flight; no other is begun
        copies = false;
        late = true;
        if (lane == 0) atomicOr(a.err_word, kErrTimeout);
      }
    }
    if (here) {
      phase ^= 1;
#pragma unroll
      for (int i = 0; i < RD::kIters; ++i) v[i] = buf[i * 32 + lane];
      __syncwarp();
    } else {
      const RowData<T> rd{static_cast<const T*>(a.logits) + row * a.ld, a.V, a.aligned != 0};
#pragma unroll
      for (int i = 0; i < RD::kIters; ++i) v[i] = rd.raw(RD::at(seg, i));
    }
    if (by_copy(it + step)) fetch(it + step);
    const RowParams P = a.params[row];
    float mx = -INFINITY;
    constexpr int kLanes = kGroup / RD::N;  // lanes of a group
    float* gmax = a.group_max + ((int64_t)row * a.segs + seg) * kGroupsPerSeg;
#pragma unroll
    for (int i = 0; i < RD::kIters; ++i) {
      float g = Vec<T>::max(v[i]);
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
      if (lane % kLanes == 0) gmax[i * (32 / kLanes) + lane / kLanes] = g;
      mx = max_nan(mx, g);
    }
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float zm = __fmul_rn(mx, P.inv_t);
    uint64_t sum = 0;
    if (zm > -INFINITY && zm < INFINITY) {  // else the row has no token, or this part no mass
      if (sums_masses(P, a.V)) {
        const Mass mass(P.inv_t, zm, table);
#pragma unroll
        for (int i = 0; i < RD::kIters; ++i) {
          float x[RD::N];
          Vec<T>::unpack(v[i], x);
#pragma unroll
          for (int e = 0; e < RD::N; ++e) sum = mass.add(sum, mass.z(x[e]));
        }
        sum = warp_sum_u64(sum);
      } else if (a.out_logprobs) {
        // (for log-probs alone, so by the special function unit, each within 2^-22: no
        // token depends on them)
        float s = 0.f;
        const float shift = lse_shift(zm), base = lse_base(zm);
#pragma unroll
        for (int i = 0; i < RD::kIters; ++i) {
          float x[RD::N];
          Vec<T>::unpack(v[i], x);
#pragma unroll
          for (int e = 0; e < RD::N; ++e)
            s += ex2_approx(__fmaf_rn(__fsub_rn(__fmul_rn(x[e], P.inv_t), shift), kLog2e, -base));
        }
        sum = __float_as_uint(warp_sum_f(s));
      }
    }
    if (lane == 0) {
      a.seg_max[(int64_t)row * a.segs + seg] = mx;
      a.seg_sum[(int64_t)row * a.segs + seg] = sum;
    }
  }
  // no copy is in flight when the CTA's memory goes to another
  if (late) mbar_wait_clocked(&bars[warp], phase, 200000000ll);
}

// ---- finishing a row ---------------------------------------------------------

// A CTA's mailboxes: slot r is written by CTA r of its team before a team barrier
// and read here after it, so that no reader waits on remote loads.  Each field
// serves one exchange, or exchanges with another barrier between the reading of
// one and the writing of the next.
struct Mail {
  uint64_t mass[kMaxCtas], all[kMaxCtas], kept[kMaxCtas];
  int count[kMaxCtas], total[kMaxCtas], tie[kMaxCtas];
  int last[kMaxCtas];  // last segment with a kept element, or -1
  Cut cut;  // from the leader
  int ok;
};

// A row's candidates are 64-bit entries: ord_key of the tempered value above the
// complement of the index, so that a larger entry is earlier in the order (z
// descending, index ascending), and a larger low half earlier in the vocabulary.
__device__ __forceinline__ uint64_t entry_of(float z, int j) {
  return ((uint64_t)ord_key(z) << 32) | (uint32_t)~j;
}
__device__ __forceinline__ float entry_z(uint64_t e) { return key_value((uint32_t)(e >> 32)); }
__device__ __forceinline__ int entry_index(uint64_t e) { return (int)~(uint32_t)e; }

struct Hist {
  uint32_t own[kBins];
  uint32_t sum[kBins];  // over the team
};

struct Shared {
  Mail mail;
  float red_f[kWarpsF];
  uint64_t red_w[kWarpsF], red_n[kWarpsF];
  int red_i[kWarpsF];
  uint2 table[kTable];
  float seg_max[kMaxSegs];    // raw maxima of the row's segments
  uint64_t seg_w[kMaxSegs];   // their masses (element units), then inclusive sums
  int seg_n[kMaxSegs];        // candidates of the segments, then those before each
  int lo, hi;
  float least[3];             // thresholds on raw logits
  int bin;
  uint32_t bin_n;
  uint64_t above;
  uint32_t digit_n[256];      // radix selection, 8 bits at a time
  unsigned long long digit_w[256];
  uint64_t run[kThreadsF];  // inclusive masses of the threads' list entries
  union {
    uint64_t found[kList];  // candidates, in any order
    uint16_t groups[kMaxSegs * kGroupsPerSeg / 2];  // groups to read, in order
  };
  // (the list lies over hist.own; its buckets are in hist.sum)
  union alignas(16) {
    Hist hist;
    uint64_t list[kList];  // candidates put in order
  };
};

// This CTA's shared memory, by its own name: a reference handed into a function
// that is not inlined would make every access, and every atomic, a generic one.
__device__ __forceinline__ Shared& smem() {
  extern __shared__ __align__(128) unsigned char dyn[];
  return *reinterpret_cast<Shared*>(dyn);
}

// A row and the CTAs that finish it (a team: the cluster, or rank 0 alone).
template <typename T>
struct Row {
  RowData<T> rd;
  Mass mass;
  float mx, m;  // maximum, tempered maximum
  int segs;     // of the row
  int drop;     // row sums are in units of 2^(E - kElemBits + drop)
  int C, rank;  // the team
  int s0, s1;   // this CTA's segments
  int per;      // segments to a CTA
  __device__ __forceinline__ Row(const RowData<T>& rd_, const Mass& mass_, float mx_, float m_,
                                 int segs_, int drop_, int C_, int rank_)
      : rd(rd_), mass(mass_), mx(mx_), m(m_), segs(segs_), drop(drop_), C(C_), rank(rank_) {
    per = (segs + C - 1) / C;
    s0 = min(segs, rank * per);
    s1 = min(segs, s0 + per);
  }
  __device__ __forceinline__ Shared* at(int r) {
    return C > 1 ? cg::this_cluster().map_shared_rank(&smem(), r) : &smem();
  }
  __device__ __forceinline__ void sync() {
    if (C > 1) cg::this_cluster().sync();
    else __syncthreads();
  }
  // thread r of the block stores v in this CTA's slot of CTA r's mailbox
  template <typename V>
  __device__ __forceinline__ void send(V (Mail::*field)[kMaxCtas], V v) {
    if ((int)threadIdx.x < C) (at((int)threadIdx.x)->mail.*field)[rank] = v;
  }
  __device__ __forceinline__ uint64_t coarse(uint64_t w) const {
    return (w + (1ull << (drop - 1))) >> drop;
  }
  __device__ __forceinline__ float seg_top(int s) const { return mass.z(smem().seg_max[s]); }
};

// Linear bins of the logits below `top` (no logit above it is asked for): a fixed
// number to a logit, whatever the temperature.
struct Bins {
  float per, top_bins;
  __device__ __forceinline__ Bins(float top, float per_) {
    per = per_;
    top_bins = __fmul_rn(top, per_);
  }
  // distance below the top in bins
  __device__ __forceinline__ float dist(float x) const { return __fmaf_rn(x, -per, top_bins); }
  // kMagic + the number of the bin, as a float; the last bin has no end
  __device__ __forceinline__ float bin_f(float x) const {
    return __fadd_rn(fminf(dist(x), (float)(kBins - 1)), kMagic);
  }
};
__device__ __forceinline__ int bin_no(float bin_f) {
  return __float_as_int(bin_f) - __float_as_int(kMagic);
}

// The thread's kBins / kThreadsF neighbouring bins.
__device__ __forceinline__ void load_bins(const uint32_t* bins, uint32_t (&c)[kBins / kThreadsF]) {
  static_assert(kBins / kThreadsF == 8, "two 16-byte loads");
  const uint4* p = reinterpret_cast<const uint4*>(bins) + threadIdx.x * 2;
  const uint4 a = p[0], b = p[1];
  c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
  c[4] = b.x, c[5] = b.y, c[6] = b.z, c[7] = b.w;
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
  for (int i = 0; i < kWarpsF; ++i) {
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
  for (int i = 0; i < kWarpsF; ++i) v += sh.red_f[i];
  return v;
}
__device__ __forceinline__ int block_sum(Shared& sh, int v) {
  v = warp_sum_i(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.red_i[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kWarpsF; ++i) v += sh.red_i[i];
  return v;
}

// The smallest logit x whose tempered value z(x) satisfies `reaches`, a predicate
// that holds from some z on: a search of the order keys, 32 at a time.  One warp.
template <typename F>
__device__ __forceinline__ float least_logit(const Mass& mass, F reaches) {
  const uint32_t lane = threadIdx.x & 31;
  uint32_t lo = 0;  // the answer is at or above
#pragma unroll 1
  for (int shift = 27; shift >= -3; shift -= 5) {
    const uint32_t step = shift > 0 ? 1u << shift : 1u;
    const uint32_t key = lo + lane * step + (step - 1);  // the last of the lane's share
    const float x = key_value(key);
    // (NaN keys lie below -inf and above +inf)
    const bool yes = key >= lo && (key >= 0xff800000u || (key >= 0x007fffffu && reaches(mass.z(x))));
    const unsigned no = __popc(__ballot_sync(0xffffffffu, !yes));
    if (no == 32) return INFINITY;
    lo += no * step;
  }
  return key_value(lo);
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
// any number of equal elements: the way of last resort.  A warp whose elements
// fall on one digit adds them up first (equal values would all go to one address).
//   MASS: elements are kept while the mass before them is <= target.
//   else: the first `target` of them are kept (1 <= target <= their number).
// Every CTA of the team returns the same cut.
template <typename T, bool MASS>
__device__ __noinline__ Cut radix_select(const Row<T>& row_in, Cut cut, uint64_t target) {
  Row<T> rw = row_in;  // in registers
  rw.mass.table = smem().table;
  using RD = RowData<T>;
  Shared& sh = smem();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t prefix = 0;
  uint64_t before = 0;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) {
      sh.digit_n[tid] = 0;
      sh.digit_w[tid] = 0;
    }
    rw.sync();
    for (int s = rw.s0 + warp; s < rw.s1; s += kWarpsF) {
      if (rw.seg_top(s) < cut.z) continue;
#pragma unroll 1
      for (int i = 0; i < RD::kIters; ++i) {
        const int at = RD::at(s, i);
        float x[RD::N];
        rw.rd.load(at, x);
#pragma unroll 1
        for (int e = 0; e < RD::N; ++e) {
          const float z = rw.mass.z(x[e]);
          const uint32_t k = ord_key(z);
          const bool in = cut.keeps(z, at + e) && (shift == 24 || (k >> (shift + 8)) == prefix);
          const int bin = (k >> shift) & 255;
          const unsigned ins = __ballot_sync(0xffffffffu, in);
          if (!ins) continue;
          const uint64_t w = MASS && in ? rw.coarse(rw.mass.of(z)) : 0;
          const int first = __shfl_sync(0xffffffffu, bin, __ffs(ins) - 1);
          if (__all_sync(0xffffffffu, !in || bin == first)) {
            const uint64_t sum = MASS ? warp_sum_u64(w) : 0;
            if (lane == 0) {
              atomicAdd(&sh.digit_n[first], (unsigned)__popc(ins));
              if (MASS && sum) atomicAdd(&sh.digit_w[first], (unsigned long long)sum);
            }
          } else if (in) {
            atomicAdd(&sh.digit_n[bin], 1u);
            if (MASS && w) atomicAdd(&sh.digit_w[bin], (unsigned long long)w);
          }
        }
      }
    }
    __syncthreads();
    // the others' digits are added to the leader's, which finds the boundary
    if (rw.rank != 0 && tid < 256 && sh.digit_n[tid]) {
      atomicAdd(&rw.at(0)->digit_n[tid], sh.digit_n[tid]);
      if (MASS) atomicAdd(&rw.at(0)->digit_w[tid], sh.digit_w[tid]);
    }
    rw.sync();
    if (rw.rank == 0 && warp == 0) find_digit<MASS>(sh, before, target);
    rw.sync();
    const Shared* lead = rw.at(0);
    prefix = (prefix << 8) | (uint32_t)lead->bin;
    before = lead->above;
  }
  const uint32_t ties = rw.at(0)->bin_n;
  rw.sync();
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
  for (int s = rw.s0 + warp; s < rw.s1; s += kWarpsF) {
    int c = 0;
    if (rw.seg_top(s) >= zk) {
#pragma unroll 1
      for (int i = 0; i < RD::kIters; ++i) {
        const int at = RD::at(s, i);
        float x[RD::N];
        rw.rd.load(at, x);
#pragma unroll
        for (int e = 0; e < RD::N; ++e) c += rw.mass.z(x[e]) == zk && at + e <= old_idx;
      }
      c = warp_sum_i(c);
    }
    if (lane == 0) {
      sh.seg_n[s] = c;
      mine += c;
    }
  }
  mine = block_sum(sh, mine);
  rw.send(&Mail::total, mine);
  rw.sync();
  uint64_t ahead = 0;
  for (int r = 0; r < rw.rank; ++r) ahead += sh.mail.total[r];
  if (tid == 0) sh.lo = -1;
  __syncthreads();
  if (take > ahead && take <= ahead + mine && warp == 0) {
    int left = (int)(take - ahead), s = rw.s0;
    while (left > sh.seg_n[s]) left -= sh.seg_n[s++];
    for (int i = 0; i < RD::kIters && left > 0; ++i) {
      const int at = RD::at(s, i);
      float x[RD::N];
      rw.rd.load(at, x);
      int c = 0;
#pragma unroll
      for (int e = 0; e < RD::N; ++e) c += rw.mass.z(x[e]) == zk && at + e <= old_idx;
      const int inc = warp_scan(c);
      if (left > inc - c && left <= inc) {
        int nth = left - (inc - c);
#pragma unroll
        for (int e = 0; e < RD::N; ++e)
          if (rw.mass.z(x[e]) == zk && --nth == 0) sh.lo = at + e;
      }
      left -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  rw.send(&Mail::tie, sh.lo);
  rw.sync();
  int idx = -1;
  for (int r = 0; r < rw.C; ++r) idx = max(idx, sh.mail.tie[r]);
  return Cut{zk, idx};
}

constexpr int kListDrop = 2;  // list masses: units of 2^(E - kElemBits + 2), 2048 below 2^62

// found[0, n) into list, by value (the order of the entries) or by index.  Up to
// 512: every entry counts those ahead of it, the comparisons shared out over all
// threads.  Beyond: into 4096 buckets, then each entry counts those ahead of it in
// its bucket.  (A bitonic sort of 1400 entries with few equal ones took 25 000
// cycles, this takes 10 000.)
template <bool BY_INDEX>
__device__ __noinline__ void order_entries(int n, int V) {
  Shared& sh = smem();
  const int tid = threadIdx.x;
  auto ahead_of = [](uint64_t e, uint64_t of) {
    return BY_INDEX ? (uint32_t)e > (uint32_t)of : e > of;
  };
  __syncthreads();
  if (n <= kThreadsF) {
    int parts = 1;  // threads that share an entry: neighbours, at most a warp
    while (parts < 32 && 2 * parts * n <= kThreadsF) parts *= 2;
    const int i = tid / parts, part = tid % parts;
    const uint64_t mine = i < n ? sh.found[i] : 0ull;
    int ahead = 0;
    if (i < n)
      for (int j = part; j < n; j += parts) ahead += ahead_of(sh.found[j], mine);
    for (int o = 1; o < parts; o *= 2) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    if (i < n && part == 0) sh.list[ahead] = mine;
    __syncthreads();
    return;
  }
  constexpr int kPer = kBins / kThreadsF;
  uint64_t e[kListPerThread];
  uint64_t most = 0, least = ~0ull;
#pragma unroll
  for (int q = 0; q < kListPerThread; ++q) {
    const int i = tid + q * kThreadsF;
    e[q] = i < n ? sh.found[i] : 0ull;
    if (i < n) {
      most = max(most, e[q]);
      least = min(least, e[q]);
    }
  }
  float top = 0.f, per = 0.f;
  if (!BY_INDEX) {  // the buckets span the entries' own values
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(most >> 32));
    const uint32_t lo = __reduce_min_sync(0xffffffffu, (uint32_t)(least >> 32));
    if ((tid & 31) == 0) {
      sh.red_w[tid >> 5] = hi;
      sh.red_n[tid >> 5] = lo;
    }
    __syncthreads();
    uint64_t a = 0, b = ~0ull;
    for (int i = 0; i < kWarpsF; ++i) {
      a = max(a, sh.red_w[i]);
      b = min(b, sh.red_n[i]);
    }
    top = key_value((uint32_t)a);
    per = (float)(kBins - 1) / fmaxf(top - key_value((uint32_t)b), 1e-30f);
  }
  int shift = 0;
  while (((V - 1) >> shift) >= kBins) ++shift;
  auto bucket_of = [&](uint64_t e) {
    return BY_INDEX ? entry_index(e) >> shift
                    : (int)fminf(fmaxf((top - entry_z(e)) * per, 0.f), (float)(kBins - 1));
  };
  uint32_t* bucket = sh.hist.sum;
#pragma unroll
  for (int q = 0; q < kPer; ++q) bucket[tid + q * kThreadsF] = 0;
  __syncthreads();
  int at[kListPerThread];
#pragma unroll
  for (int q = 0; q < kListPerThread; ++q) {
    const int i = tid + q * kThreadsF;
    at[q] = i < n ? (int)atomicAdd(&bucket[bucket_of(e[q])], 1u) : 0;
  }
  __syncthreads();
  uint32_t c[kPer];
  uint64_t sum = 0, all;
  load_bins(bucket, c);
#pragma unroll
  for (int q = 0; q < kPer; ++q) sum += c[q];
  uint32_t begin = (uint32_t)block_scan(sh, sum, &all);
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    bucket[tid * kPer + q] = begin;
    begin += c[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kListPerThread; ++q)
    if (tid + q * kThreadsF < n) sh.list[bucket[bucket_of(e[q])] + at[q]] = e[q];
  __syncthreads();
#pragma unroll 1
  for (int q = 0; q < kListPerThread; ++q) {
    if (tid + q * kThreadsF >= n) break;
    const uint64_t mine = q == 0 ? e[0] : q == 1 ? e[1] : q == 2 ? e[2] : e[3];
    const int b = bucket_of(mine), from = bucket[b], to = b + 1 < kBins ? bucket[b + 1] : n;
    int place = from;
    for (int i = from; i < to; ++i) place += ahead_of(sh.list[i], mine);
    at[0] = q == 0 ? place : at[0];
    at[1] = q == 1 ? place : at[1];
    at[2] = q == 2 ? place : at[2];
    at[3] = q == 3 ? place : at[3];
  }
  static_assert(kListPerThread == 4, "the entries of a thread above");
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kListPerThread; ++q)
    if (tid + q * kThreadsF < n) sh.list[at[q]] = e[q];
  __syncthreads();
}
// The cut whose last element is entry i of the list.
__device__ __forceinline__ Cut sorted_cut(const Shared& sh, int i) {
  return Cut{entry_z(sh.list[i]), entry_index(sh.list[i])};
}
// Of the first n entries of the list, those with a mass (list units) of at most
// target before them: the cut, and the mass of all n in *all.  `share` >= 0: the
// target is that part of it instead.
__device__ __forceinline__ Cut cut_by_mass(Shared& sh, const Mass& mass, int n, uint64_t target,
                                           float share, uint64_t* all) {
  const int tid = threadIdx.x;
  uint64_t w[kListPerThread], sum = 0;
#pragma unroll
  for (int q = 0; q < kListPerThread; ++q) {
    const int i = tid * kListPerThread + q;
    w[q] = i < n ? (mass.of(entry_z(sh.list[i])) + 2) >> kListDrop : 0;
    sum += w[q];
  }
  uint64_t a = block_scan(sh, sum, all);
  if (share >= 0.f) target = part_of(*all, share);
  int kept = 0;
#pragma unroll
  for (int q = 0; q < kListPerThread; ++q) {
    kept += tid * kListPerThread + q < n && a <= target;
    a += w[q];
  }
  kept = block_sum(sh, kept);
  return sorted_cut(sh, kept - 1);
}

// The lanes' marked elements (bit e of `take`: element at + e) to the CTA's found
// entries, counted in sh.bin.  Whole warp.
template <typename T>
__device__ __forceinline__ void append(Shared& sh, const RowData<T>& rd, const Mass& mass, int at,
                                       unsigned take) {
  if (!__any_sync(0xffffffffu, take)) return;
  const int c = __popc(take);
  const int inc = warp_scan(c);
  int q = 0;
  if ((threadIdx.x & 31) == 31) q = atomicAdd(&sh.bin, inc);
  q = __shfl_sync(0xffffffffu, q, 31) + inc - c;
#pragma unroll 1
  for (; take; take &= take - 1, ++q) {
    const int j = at + __ffs(take) - 1;
    if (q < kList) sh.found[q] = entry_of(mass.z(elem(rd.data[j])), j);
  }
}

// The boundary of the elements kept by `cut` by linear histograms, which bracket
// it closer and closer, and a list of the elements in the bracket, once it holds
// them.  One histogram over the row nearly always does; the masses above a
// bracket are summed exactly before the next is made of it.
//   MASS: elements are kept while the mass before them is <= target (row units);
//   those below z_least have too little mass for the boundary to be among them.
//   On success the CTAs' seg_w hold the masses of the kept elements (element units).
//   else: the first `target` of them are kept (z_least: -inf).
// PLAIN: `cut` has no index, so that a threshold on the logits says it all.
// Returns false (the same in every CTA) when too many elements are equal, or, by
// mass, when a bracket turns out not to hold the boundary.
template <typename T, bool MASS, bool PLAIN>
__device__ __noinline__ bool band_select(const Row<T>& row_in, Cut* cut_io, uint64_t target,
                                         float z_least) {
  Row<T> rw = row_in;  // in registers
  rw.mass.table = smem().table;
  using RD = RowData<T>;
  Shared& sh = smem();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Cut cut = *cut_io;
  constexpr int kPer = kBins / kThreadsF;
  __syncthreads();
  if (warp == 0) {
    const float least = fmaxf(cut.z, z_least);
    const float x = least_logit(rw.mass, [&](float z) { return z >= least; });
    if (lane == 0) sh.least[0] = x;
  }
  __syncthreads();
  float x_from = sh.least[0], x_to = INFINITY;  // the bracket: x_from <= x < x_to
  // (by mass: bins narrow enough for the quadratic below)
  float per = MASS ? fmaxf(kBinsPerLogit, 16.f * rw.mass.inv_t) : kBinsPerLogit;
  // (edges off the grid that bf16 logits lie on: a value on an edge would fall
  // to either side)
  float top = rw.mx + 0.3f / per;
  uint64_t above = 0;  // mass (or elements) above the bracket
  int n = 0;
#pragma unroll 1
  for (int level = 0;; ++level) {
    const Bins bins(top, per);
#pragma unroll
    for (int q = 0; q < kPer; ++q) sh.hist.own[tid + q * kThreadsF] = 0;
    if (tid == 0) {
      sh.lo = kBins;
      sh.hi = -1;
    }
    __syncthreads();
    // by mass: each element adds its mass relative to its bin's middle in units of
    // 1/4063, so a bin's mass is known to within 1.3e-4 of itself
    const float nats = rw.mass.inv_t / per;  // to a bin
    const float c1 = -4063.f * nats, c2 = 4063.f * 0.5f * nats * nats;
    for (int s = rw.s0 + warp; s < rw.s1; s += kWarpsF) {
      if (sh.seg_max[s] < x_from) continue;
      each_vector(rw.rd, s, [&](const float(&x)[RD::N], int at) {
#pragma unroll
        for (int e = 0; e < RD::N; ++e) {
          const float t = bins.dist(x[e]);
          bool in = x[e] >= x_from && x[e] < x_to;
          if (!PLAIN) in = in && cut.keeps(rw.mass.z(x[e]), at + e);
          if (MASS) {  // 4063 e^(-f nats), f in [-1/2, 1/2], through a rounding by 2^23
            const float b = __fadd_rn(t, kMagic);
            const float f = __fsub_rn(t, __fsub_rn(b, kMagic));
            const uint32_t add =
                __float_as_uint(__fmaf_rn(f, __fmaf_rn(f, c2, c1), 8388608.f + 4063.f)) & 0x1fffu;
            if (in && t < (float)(kBins - 1)) atomicAdd(&sh.hist.own[max(bin_no(b), 0)], add);
          } else {
            if (in) atomicAdd(&sh.hist.own[max(bin_no(bins.bin_f(x[e])), 0)], 1u);
          }
        }
      });
    }
    // the team's histogram: CTA r sums a share of the bins and sends it to all
    rw.sync();
    const uint32_t* from = sh.hist.own;
    if (rw.C > 1) {
      const int share = kBins / rw.C;
      for (int q = tid; q < share; q += kThreadsF) {
        const int bin = rw.rank * share + q;
        uint32_t c = 0;
#pragma unroll 4
        for (int r = 0; r < rw.C; ++r) c += rw.at(r)->hist.own[bin];
#pragma unroll 4
        for (int r = 0; r < rw.C; ++r) rw.at(r)->hist.sum[bin] = c;
      }
      rw.sync();
      from = sh.hist.sum;
    }
    uint32_t cn[kPer];
    load_bins(from, cn);
    if (MASS) {
      float cf[kPer], tf = 0.f;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        cf[q] = (float)cn[q] * ex2_approx((float)(tid * kPer + q) * (-kLog2e * nats));
        tf += cf[q];
      }
      const float inc = warp_scan(tf);
      if (lane == 31) sh.red_f[warp] = inc;
      __syncthreads();
      float a = inc - tf;
      for (int i = 0; i < kWarpsF; ++i)
        if (i < warp) a += sh.red_f[i];
      constexpr float kSlack = 1.f / 6144;  // of the bins' masses and their fp32 sums
      // the target in the histogram's units (4063 of the mass at `top`)
      const float want = __ull2float_rn(target - above) * 4063.f /
                         exp2f(__fmaf_rn(rw.mass.z(top) - rw.mass.c, kLog2e,
                                         (float)(kElemBits - rw.drop - rw.mass.E())));
      int lo = kBins, hi = -1;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (cn[q] > 0) {
          // bins that end before the target are kept whole, those that begin
          // after it not at all
          if (a + cf[q] >= want * (1.f - kSlack)) lo = min(lo, tid * kPer + q);
          if (a <= want * (1.f + kSlack)) hi = tid * kPer + q;
        }
        a += cf[q];
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (lane == 0) {
        atomicMin(&sh.lo, lo);
        atomicMax(&sh.hi, hi);
      }
    } else {
      uint64_t tn = 0, unused;
#pragma unroll
      for (int q = 0; q < kPer; ++q) tn += cn[q];
      uint64_t a = above + block_scan(sh, tn, &unused);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (a < target && a + cn[q] >= target) sh.lo = sh.hi = tid * kPer + q;
        a += cn[q];
      }
    }
    __syncthreads();
    const int lo = sh.lo, hi = sh.hi;
    if (lo > hi) return false;  // (a histogram without mass)

    // the new bracket, by tempered values: the elements from the far edge of bin
    // hi up to the near edge of bin lo
    const float near = top - ((float)lo - 0.5f) / per, far = top - ((float)hi + 0.5f) / per;
    if (warp == 1 || warp == 2) {
      const float edge = rw.mass.z(warp == 1 ? near : far);
      const float x = least_logit(rw.mass, [&](float z) { return z > edge; });
      if (lane == 0) sh.least[warp] = x;
    }
    if (tid == 0) sh.bin = 0;  // entries so far
    __syncthreads();
    const float x_up = lo == 0 ? x_to : fminf(fmaxf(sh.least[1], x_from), x_to);
    const float x_band = hi == kBins - 1 ? x_from : fmaxf(sh.least[2], x_from);
    // the masses (or number) above it, and its elements into this CTA's entries;
    // segments that end below it are not read
    uint64_t more = 0;
    for (int s = rw.s0 + warp; s < rw.s1; s += kWarpsF) {
      uint64_t up_w = 0;
      if (sh.seg_max[s] >= x_band) {
        each_vector(rw.rd, s, [&](const float(&x)[RD::N], int at) {
          unsigned take = 0;
#pragma unroll
          for (int e = 0; e < RD::N; ++e) {
            const float z = rw.mass.z(x[e]);
            bool in = x[e] < x_to;
            if (!PLAIN) in = in && cut.keeps(z, at + e);
            const bool up = x[e] >= x_up && in;
            take |= x[e] >= x_band && in && !up ? 1u << e : 0u;
            // (a select, not a branch: the masses of a vector overlap.  Going through
            // the lanes' marked elements alone is 9 % slower at p = 0.9.)
            if (MASS) up_w = rw.mass.add(up_w, up ? z : -INFINITY);
            else up_w += up;
          }
          append(sh, rw.rd, rw.mass, at, take);
        });
        up_w = warp_sum_u64(up_w);
      }
      if (lane == 0) {
        if (MASS) sh.seg_w[s] = level > 0 ? sh.seg_w[s] + up_w : up_w;
        more += MASS ? rw.coarse(up_w) : up_w;
      }
    }
    if (lane == 0) sh.red_w[warp] = more;
    __syncthreads();
    rw.send(&Mail::count, sh.bin);
    if (warp == 0) rw.send(&Mail::mass, (uint64_t)warp_sum_u64(lane < kWarpsF ? sh.red_w[lane] : 0));
    rw.sync();
    n = 0;
    int base = 0;
    for (int r = 0; r < rw.C; ++r) {
      if (r == rw.rank) base = n;
      n += sh.mail.count[r];
      above += sh.mail.mass[r];
    }
    if (MASS ? above > target : above >= target) return false;  // the boundary is above it
    if (n <= kList) {
      if (rw.rank > 0) {  // behind the leader's own, in any order
        const int own = sh.mail.count[rw.rank];
        uint64_t* to = rw.at(0)->found + base;
        for (int i = tid; i < own; i += kThreadsF) to[i] = sh.found[i];
      }
      rw.sync();
      if (n == 0) return false;
      break;
    }
    rw.sync();
    if (level == 3) return false;
    x_from = x_band;
    x_to = x_up;
    top = fminf(near, top);
    // (the last bin has no end: the next bins begin where it does)
    if (hi < kBins - 1) per *= (float)(kBins - 2) / (float)(hi - lo + 1);
  }
  if (rw.rank == 0) {
    bool ok = true;
    Cut found{0.f, kMaxIdx};
    order_entries<false>(n, rw.rd.V);
    if (MASS) {
      // the boundary lies in the bracket: the mass above it is within the
      // target, that at its end is not
      ok = (target - above) < (1ull << (62 - rw.drop));
      const uint64_t left = ok ? (target - above) << (rw.drop - kListDrop) : 0;
      uint64_t band;
      found = cut_by_mass(sh, rw.mass, n, left, -1.f, &band);
      ok = ok && left < band;
      if (ok)
        for (int i = tid; i < n; i += kThreadsF) {
          const int j = entry_index(sh.list[i]);
          const float z = entry_z(sh.list[i]);
          if (found.keeps(z, j))
            atomicAdd((unsigned long long*)&rw.at(j / kSeg / rw.per)->seg_w[j / kSeg],
                      (unsigned long long)rw.mass.of(z));
        }
    } else {
      ok = target - above <= (uint64_t)n;
      found = sorted_cut(sh, ok ? (int)(target - above) - 1 : 0);
    }
    if (tid < rw.C) {
      rw.at(tid)->mail.cut = found;
      rw.at(tid)->mail.ok = ok;
    }
  }
  rw.sync();
  const bool ok = sh.mail.ok;
  if (ok) *cut_io = sh.mail.cut;
  return ok;
}

// The top-p boundary of a bf16 row that nothing else cuts, by counting its values:
// every element of one bf16 pattern has one mass, so a slot per pattern below the
// maximum (code16; the magnitudes below 2^-12 share one, summed element by element)
// gives the masses of all prefixes exactly, without a list or a second look at a
// bracket.  A second pass adds up the kept elements' masses by segment, from a
// table of the slots'.  (256 rows of 151,936 with p = 0.99: 249 us by band_select,
// 196 so; one row 71 and 52.)  What bounds it: the shared memory's atomics of the
// first pass and lookups of the second, about 9 cycles a warp each.
//   target as in band_select; *cut_io gets this CTA's own view of the cut: of the
//   elements at the boundary, which are kept by index, its own up to idx.
// Returns false (the same in every CTA) when the boundary is in the shared slot or
// past the last slot, or when tempering could make two patterns equal.
template <typename T>
__device__ __noinline__ bool code_select(const Row<T>& row_in, Cut* cut_io, uint64_t target) {
  Row<T> rw = row_in;  // in registers
  rw.mass.table = smem().table;
  using RD = RowData<T>;
  Shared& sh = smem();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kBins == kCodeSlots, "a slot to a bin");
  constexpr int kPer = kBins / kThreadsF;
  const int top = code16(__float_as_uint(rw.mx) >> 16);
  if (top == 0 || !(rw.mass.inv_t > 0x1p-64f) || !(fabsf(rw.m) < INFINITY)) return false;
  auto slot_of = [&](float x) { return top - code16(__float_as_uint(x) >> 16); };
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPer; ++q) sh.hist.own[tid + q * kThreadsF] = 0;
  if (tid == 0) {
    sh.digit_w[0] = 0;  // mass of the shared slot, row units
    sh.hi = -1;
  }
  rw.sync();
  uint64_t shared_w = 0;
  for (int s = rw.s0 + warp; s < rw.s1; s += kWarpsF) {
    each_vector(rw.rd, s, [&](const float(&x)[RD::N], int) {
#pragma unroll
      for (int e = 0; e < RD::N; ++e) {
        const int slot = slot_of(x[e]);
        if (slot < kBins - 1) atomicAdd(&sh.hist.own[slot], 1u);
        if (slot == top) shared_w += rw.coarse(rw.mass.of(rw.mass.z(x[e])));
      }
    });
  }
  shared_w = warp_sum_u64(shared_w);
  if (lane == 0 && shared_w) atomicAdd(&rw.at(0)->digit_w[0], (unsigned long long)shared_w);
  // the team's counts: CTA r sums a share of the slots and sends it to all
  rw.sync();
  const uint32_t* from = sh.hist.own;
  if (rw.C > 1) {
    const int share = kBins / rw.C;
    for (int q = tid; q < share; q += kThreadsF) {
      const int slot = rw.rank * share + q;
      uint32_t c = 0;
#pragma unroll 4
      for (int r = 0; r < rw.C; ++r) c += rw.at(r)->hist.own[slot];
#pragma unroll 4
      for (int r = 0; r < rw.C; ++r) rw.at(r)->hist.sum[slot] = c;
    }
    if (rw.rank > 0 && tid == 0) sh.digit_w[0] = rw.at(0)->digit_w[0];
    rw.sync();
    from = sh.hist.sum;
  }
  // a slot's element (over the counts, once they are read) and its mass in row units
  uint32_t cn[kPer];
  load_bins(from, cn);
  static_assert(sizeof(sh.hist) >= kBins * sizeof(uint64_t), "a mass for every slot");
  uint64_t* table = reinterpret_cast<uint64_t*>(&sh.hist);
  __syncthreads();
  uint64_t row_w[kPer], sum = 0, all;
#pragma unroll
  for (int q = 0; q < kPer; q += 2) {
    uint64_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int slot = tid * kPer + q + i;
      w[i] = slot != top ? rw.mass.of(rw.mass.z(code_value(top - slot))) : 0;
      // cn * w + half a row unit, in 128 bits
      const uint64_t n = cn[q + i], lo = n * w[i], half = 1ull << (rw.drop - 1);
      const uint64_t hi = __umul64hi(n, w[i]) + (lo + half < lo);
      row_w[q + i] = (hi << (64 - rw.drop)) | ((lo + half) >> rw.drop);
      if (slot == top) row_w[q + i] = sh.digit_w[0];
      sum += row_w[q + i];
    }
    *reinterpret_cast<ulonglong2*>(table + tid * kPer + q) = make_ulonglong2(w[0], w[1]);
  }
  uint64_t a = block_scan(sh, sum, &all);
  int mine = -1;
  uint64_t mine_a = 0;
  uint32_t mine_n = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (cn[q] && a <= target) {
      mine = tid * kPer + q;
      mine_a = a;
      mine_n = cn[q];
    }
    a += row_w[q];
  }
  const int last = __reduce_max_sync(0xffffffffu, mine);
  if (lane == 0) atomicMax(&sh.hi, last);
  __syncthreads();
  if (mine >= 0 && mine == sh.hi) {
    sh.above = mine_a;
    sh.bin_n = mine_n;
  }
  __syncthreads();
  const int edge = sh.hi;
  if (edge < 0 || edge == top || all <= target) return false;
  const uint64_t w_edge = table[edge], n_edge = sh.bin_n, left = target - sh.above;
  if (left >= (1ull << (62 - rw.drop)) || w_edge == 0) return false;
  const uint64_t take = min((left << rw.drop) / w_edge + 1, n_edge);  // of the equal elements
  const float x_edge = code_value(top - edge);
  int ties_all = 0;
  for (int s = rw.s0 + warp; s < rw.s1; s += kWarpsF) {
    uint64_t up = 0;
    int ties = 0;
    if (sh.seg_max[s] >= x_edge) {
      each_vector(rw.rd, s, [&](const float(&x)[RD::N], int) {
#pragma unroll
        for (int e = 0; e < RD::N; ++e) {
          const int slot = slot_of(x[e]);
          if (slot < edge) up += slot == top ? rw.mass.of(rw.mass.z(x[e])) : table[slot];
          ties += slot == edge;
        }
      });
      up = warp_sum_u64(up);
      ties = warp_sum_i(ties);
    }
    if (lane == 0) {
      sh.seg_w[s] = up;
      sh.seg_n[s] = ties;
      ties_all += ties;
    }
  }
  ties_all = block_sum(sh, ties_all);
  rw.send(&Mail::total, ties_all);
  rw.sync();
  uint64_t before = 0;
  for (int r = 0; r < rw.rank; ++r) before += sh.mail.total[r];
  int idx = before + ties_all <= take ? kMaxIdx : -1;  // all of this CTA's ties, or none, or
  if (warp == 0) {
    uint64_t carry = before;
    for (int b = rw.s0; b < rw.s1; b += 32) {
      const uint64_t c = b + lane < rw.s1 ? sh.seg_n[b + lane] : 0;
      const uint64_t inc = warp_scan(c) + carry, ahead = inc - c;
      const uint64_t kept = take <= ahead ? 0 : min(c, take - ahead);
      if (b + lane < rw.s1) sh.seg_w[b + lane] += kept * w_edge;
      const unsigned part = __ballot_sync(0xffffffffu, ahead < take && take < inc);
      if (part) {  // those up to the take-th, in this segment
        const int s = b + __ffs(part) - 1;
        int nth = (int)__shfl_sync(0xffffffffu, kept, __ffs(part) - 1);
        each_vector(rw.rd, s, [&](const float(&x)[RD::N], int at) {
          int n = 0;
#pragma unroll
          for (int e = 0; e < RD::N; ++e) n += slot_of(x[e]) == edge;
          const int sum = warp_scan(n);
          if (nth > sum - n && nth <= sum) {
            int k = nth - (sum - n);
#pragma unroll
            for (int e = 0; e < RD::N; ++e)
              if (slot_of(x[e]) == edge && --k == 0) idx = at + e;
          }
          nth -= __shfl_sync(0xffffffffu, sum, 31);
        });
        idx = __reduce_max_sync(0xffffffffu, idx);
      }
      carry = __shfl_sync(0xffffffffu, inc, 31);
    }
    // a boundary between two segments of this CTA: everything before the first
    // segment whose ties are not kept
    if (idx < 0 && before < take && take < before + ties_all) {
      uint64_t run = before;
      for (int s = rw.s0; s < rw.s1; ++s) {
        if (run == take) {
          idx = s * kSeg - 1;
          break;
        }
        run += sh.seg_n[s];
      }
    }
    if (lane == 0) sh.lo = idx;
  }
  __syncthreads();
  *cut_io = Cut{rw.mass.z(x_edge), sh.lo};
  return true;
}

// Masses of the kept elements by segment, into seg_w (element units).
template <typename T>
__device__ __noinline__ void kept_mass(const Row<T>& row_in, const Cut cut) {
  Row<T> rw = row_in;  // in registers
  rw.mass.table = smem().table;
  using RD = RowData<T>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (warp == 0) {
    const float least = fmaxf(cut.z, rw.m - 64.f);  // no mass below
    const float x = least_logit(rw.mass, [&](float z) { return z >= least; });
    if (lane == 0) smem().least[0] = x;
  }
  __syncthreads();
  const float x_cut = smem().least[0];
  const bool plain = cut.idx == kMaxIdx;
  for (int s = rw.s0 + warp; s < rw.s1; s += kWarpsF) {
    uint64_t w = 0;
    if (smem().seg_max[s] >= x_cut) {
      each_vector(rw.rd, s, [&](const float(&x)[RD::N], int at) {
#pragma unroll
        for (int e = 0; e < RD::N; ++e) {
          const float z = rw.mass.z(x[e]);
          const bool in = x[e] >= x_cut && (plain || cut.keeps(z, at + e));
          w = rw.mass.add(w, in ? z : -INFINITY);
        }
      });
      w = warp_sum_u64(w);
    }
    if (lane == 0) smem().seg_w[s] = w;
  }
}

// seg_w of this CTA's segments to inclusive sums in row units; returns the team's
// total, the mass of the CTAs before this one and this CTA's.  Mail::last gets the
// CTAs' last segments with an element that `cut` keeps (with an index: one of the
// elements at its value, or the end of a segment).
template <typename T>
__device__ uint64_t sum_segments(Row<T>& rw, const Cut& cut, uint64_t* before, uint64_t* own) {
  Shared& sh = smem();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (warp == 0) {
    uint64_t carry = 0;
    int last = -1;
    for (int b = rw.s0; b < rw.s1; b += 32) {
      const int s = b + lane;
      const uint64_t w = warp_scan(s < rw.s1 ? rw.coarse(sh.seg_w[s]) : (uint64_t)0) + carry;
      if (s < rw.s1) {
        sh.seg_w[s] = w;
        const float top = rw.seg_top(s);
        if (top > cut.z || (top == cut.z && cut.idx >= s * kSeg)) last = s;
      }
      carry = __shfl_sync(0xffffffffu, w, 31);
    }
    rw.send(&Mail::kept, carry);
    rw.send(&Mail::last, __reduce_max_sync(0xffffffffu, last));
  }
  rw.sync();
  uint64_t total = 0;
  for (int r = 0; r < rw.C; ++r) {
    if (r == rw.rank) *before = total;
    total += sh.mail.kept[r];
  }
  *own = sh.mail.kept[rw.rank];
  return total;
}

// The last kept element of segment s, or -1; one warp.
template <typename T>
__device__ int last_kept(const Row<T>& rw, const Cut& cut, int s, float* z_out) {
  using RD = RowData<T>;
  int idx = -1;
#pragma unroll 1
  for (int i = 0; i < RD::kIters; ++i) {
    const int at = RD::at(s, i);
    float x[RD::N];
    rw.rd.load(at, x);
    for (int e = 0; e < RD::N; ++e)
      if (cut.keeps(rw.mass.z(x[e]), at + e)) idx = at + e;
  }
  idx = __reduce_max_sync(0xffffffffu, idx);
  if (idx >= 0) *z_out = rw.mass.z(elem(rw.rd.data[idx]));
  return idx;
}

// The first kept element of this CTA whose inclusive mass (from the CTA's start)
// exceeds t (row units, below the CTA's mass); one warp.
// streamed: the segments' masses are stream_kernel's, relative to each segment's own
// maximum, and so are the elements' here: far below the row's maximum a segment has
// mass where each of its elements, relative to the row's, would have none.
template <typename T>
__device__ int find_draw(const Row<T>& rw, const Cut& cut, uint64_t t, bool streamed,
                         float* z_out) {
  using RD = RowData<T>;
  int lo = rw.s0, hi = rw.s1 - 1;  // the first segment whose inclusive mass exceeds t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (smem().seg_w[mid] > t) hi = mid;
    else lo = mid + 1;
  }
  if (lo > rw.s0) t -= smem().seg_w[lo - 1];
  Mass mass = rw.mass;
  int up = rw.drop;  // to element units
  if (streamed) {
    mass = Mass(rw.mass.inv_t, rw.seg_top(lo), rw.mass.table);
    up += rw.mass.E() - mass.E();
  }
  t = t == 0 ? 0 : t << up;
  int idx = -1;
  float zz = 0.f;
#pragma unroll 1
  for (int i = 0; i < RD::kIters; ++i) {
    const int at = RD::at(lo, i);
    float x[RD::N];
    rw.rd.load(at, x);
    uint64_t w[RD::N], sum = 0;
#pragma unroll
    for (int e = 0; e < RD::N; ++e) {
      const float z = rw.mass.z(x[e]);
      w[e] = cut.keeps(z, at + e) ? mass.of(z) : 0;
      sum += w[e];
    }
    const uint64_t inc = warp_scan(sum);
    uint64_t run = inc - sum;
    // the segment's sum was rounded to row units: a t within that of its end
    // takes the last element that has mass
    int here = -1, last = -1;
    float z_here = 0.f, z_last = 0.f;
#pragma unroll
    for (int e = 0; e < RD::N; ++e) {
      run += w[e];
      if (w[e] > 0) {
        last = at + e;
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

// Whether a filtered row is settled on the list: the whole row fits it, or the
// group maxima give a top-k row's candidates (at least twice top_k groups, so that
// the elements that reach the top_k-th maximum are not many more).
__device__ __forceinline__ bool listable(const RowParams& P, bool topk, int V) {
  if (V <= kList) return topk || (P.flags & kRowTopP);
  return topk && P.top_k <= kListTopK && 2 * P.top_k <= V / kGroup;
}

// A listable row, by one CTA: the groups that reach the top_k-th group maximum (a
// row that fits: all) hold its candidates, which go to the list; min-p, top-k and top-p are
// settled there and the draws made.  Returns false when the list does not hold
// them.
template <typename T>
__device__ __noinline__ bool draw_from_list(const Row<T>& row_in, const GivenArgs& a,
                                            const RowParams& P, const Cut minp, int top_k,
                                            int row, float ln_s) {
  Row<T> rw = row_in;  // in registers
  rw.mass.table = smem().table;
  Shared& sh = smem();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* gmax = a.group_max + (int64_t)row * rw.segs * kGroupsPerSeg;
  const int groups = rw.segs * kGroupsPerSeg;
  const Bins bins(rw.mx, kBinsPerLogit);
  constexpr int kPer = kBins / kThreadsF;
  constexpr int kHold = 8;  // neighbouring group maxima a thread holds: 4096 a round
  auto hold = [&](int b, float (&g)[kHold]) {
    const int i = b + tid * kHold;
    float4 lo = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), hi = lo;
    if (i < groups) {  // (a segment has 16 groups)
      lo = *reinterpret_cast<const float4*>(gmax + i);
      hi = *reinterpret_cast<const float4*>(gmax + i + 4);
    }
    g[0] = lo.x, g[1] = lo.y, g[2] = lo.z, g[3] = lo.w;
    g[4] = hi.x, g[5] = hi.y, g[6] = hi.z, g[7] = hi.w;
  };
  float g[kHold];
  hold(0, g);
  const bool fits = a.V <= kList;
  if (!fits) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) sh.hist.own[tid + q * kThreadsF] = 0;
    if (tid == 0) {
      sh.hi = kBins - 1;
      sh.bin_n = 0xffffffffu;  // order key of the least maximum wanted
    }
    __syncthreads();
#pragma unroll 1
    for (int b = 0; b < groups; b += kHold * kThreadsF) {
      if (b > 0) hold(b, g);
#pragma unroll
      for (int q = 0; q < kHold; ++q)
        if (g[q] > -INFINITY) atomicAdd(&sh.hist.own[max(bin_no(bins.bin_f(g[q])), 0)], 1u);
    }
    __syncthreads();
    {
      uint32_t cn[kPer];
      uint64_t tn = 0, unused;
      load_bins(sh.hist.own, cn);
#pragma unroll
      for (int q = 0; q < kPer; ++q) tn += cn[q];
      uint64_t b = block_scan(sh, tn, &unused);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (b < (uint64_t)top_k && b + cn[q] >= (uint64_t)top_k) sh.hi = tid * kPer + q;
        b += cn[q];
      }
    }
    __syncthreads();
  }
  // (fewer than top_k groups with a finite element: every finite element)
  const bool any = fits || sh.hi == kBins - 1;
  // The threshold is the least of the group maxima down to that bin: top_k groups
  // reach it, whatever the spacing of floats at that magnitude (an edge got by
  // subtracting from the row's maximum rounds back onto it from 2^17 on).
  if (!any) {
    uint32_t least = 0xffffffffu;
#pragma unroll 1
    for (int b = 0; b < groups; b += kHold * kThreadsF) {
      if (groups > kHold * kThreadsF) hold(b, g);
#pragma unroll
      for (int q = 0; q < kHold; ++q)
        if (g[q] > -INFINITY && max(bin_no(bins.bin_f(g[q])), 0) <= sh.hi)
          least = min(least, ord_key(g[q]));
    }
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) atomicMin(&sh.bin_n, least);
    __syncthreads();
  }
  if (warp == 0) {
    // by tempered values: equal ones are candidates too, they go by index
    const float edge = any ? -INFINITY : rw.mass.z(key_value(sh.bin_n));
    const float x = least_logit(rw.mass, [&](float z) { return any ? z > edge : z >= edge; });
    if (lane == 0) sh.least[0] = x;
  }
  __syncthreads();
  const float x_least = sh.least[0];
  // the groups that reach it, in order
  int n_groups = 0;
  constexpr int kCap = (int)(sizeof(sh.groups) / sizeof(sh.groups[0]));
#pragma unroll 1
  for (int b = 0; b < groups; b += kHold * kThreadsF) {
    if (groups > kHold * kThreadsF) hold(b, g);
    int c = 0;
#pragma unroll
    for (int q = 0; q < kHold; ++q) c += g[q] >= x_least;
    uint64_t all;
    int at = n_groups + (int)block_scan(sh, (uint64_t)c, &all);
#pragma unroll
    for (int q = 0; q < kHold; ++q)
      if (g[q] >= x_least) {
        if (at < kCap) sh.groups[at] = (uint16_t)(b + tid * kHold + q);
        ++at;
      }
    n_groups += (int)all;
  }
  if (n_groups > kList) return false;
  __syncthreads();
  // a warp takes kVecGroups groups with one 16-byte load a lane, in order
  constexpr int kLanes = kGroup / RowData<T>::N, kVecGroups = 32 / kLanes;
  const int rounds = (n_groups + kVecGroups - 1) / kVecGroups;
  // (out of the way of the candidates, which lie over them)
  static_assert(sizeof(sh.hist.sum) >= kList * sizeof(uint16_t), "the listed groups' room");
  uint16_t* kept_groups = reinterpret_cast<uint16_t*>(sh.hist.sum);
  constexpr int kAhead = 4;
  for (int i = tid; i < n_groups; i += kThreadsF) kept_groups[i] = sh.groups[i];
  if (tid == 0) sh.bin = 0;
  __syncthreads();
  auto place = [&](int r) {
    const int g = r * kVecGroups + lane / kLanes;
    return g < n_groups ? (int)kept_groups[g] * kGroup + (lane % kLanes) * RowData<T>::N
                        : rw.rd.V;
  };
#pragma unroll 1
  for (int r0 = warp; r0 < rounds; r0 += kWarpsF * kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) v[q] = rw.rd.raw(place(r0 + q * kWarpsF));
#pragma unroll 1
    for (int q = 0; q < kAhead; ++q) {
      float x[RowData<T>::N];
      Vec<T>::unpack(v[0], x);
      v[0] = v[1];
      v[1] = v[2];
      v[2] = v[3];
      unsigned take = 0;
#pragma unroll
      for (int e = 0; e < RowData<T>::N; ++e) take |= x[e] >= x_least ? 1u << e : 0u;
      append(sh, rw.rd, rw.mass, place(r0 + q * kWarpsF), take);
    }
  }
  __syncthreads();
  const int n = sh.bin;
  if (n < 1 || n > kList) return false;
  order_entries<false>(n, rw.rd.V);
  int kept = 0;
  for (int i = tid; i < n; i += kThreadsF) kept += entry_z(sh.list[i]) >= minp.z;
  kept = min(block_sum(sh, kept), top_k);
  uint64_t total;
  const Cut cut = P.flags & kRowTopP ? cut_by_mass(sh, rw.mass, kept, 0, P.top_p, &total)
                                     : sorted_cut(sh, kept - 1);
  order_entries<true>(n, rw.rd.V);
  // each thread holds a few neighbours of the list
  auto weight = [&](int i) -> uint64_t {
    if (i >= n) return 0;
    const float z = entry_z(sh.list[i]);
    return cut.keeps(z, entry_index(sh.list[i])) ? (rw.mass.of(z) + 2) >> kListDrop : 0;
  };
  uint64_t mine = 0;
#pragma unroll
  for (int q = 0; q < kListPerThread; ++q) mine += weight(tid * kListPerThread + q);
  const uint64_t ahead = block_scan(sh, mine, &total);
  sh.run[tid] = ahead + mine;
  __syncthreads();
  for (int d = tid; d < a.draws; d += kThreadsF) {
    const int64_t o = (int64_t)row * a.draws + d;
    const uint64_t t = part_of(total, a.uniforms[o]);
    int lo = 0, hi = kThreadsF - 1;  // the first thread whose inclusive mass exceeds t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sh.run[mid] > t) hi = mid;
      else lo = mid + 1;
    }
    uint64_t run = lo > 0 ? sh.run[lo - 1] : 0;
    int i = lo * kListPerThread;
    if (a.uniforms[o] >= 1.f)  // the last kept one, whether it has mass or not
      for (i = n - 1; i > 0 && !cut.keeps(entry_z(sh.list[i]), entry_index(sh.list[i]));) --i;
    else
      for (run += weight(i); run <= t && i + 1 < n; run += weight(i)) ++i;
    a.out_tokens[o] = entry_index(sh.list[i]);
    if (a.out_logprobs)
      a.out_logprobs[o] = __fsub_rn(__fsub_rn(entry_z(sh.list[i]), rw.m), ln_s);
  }
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreadsF, 2) finish_kernel(GivenArgs a) {
  using RD = RowData<T>;
  Shared& sh = smem();
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int row = blockIdx.x / ctas;
  const RowParams P = a.params[row];
  const bool greedy = P.flags & kRowGreedy;
  const bool topk = !greedy && P.top_k > 1 && P.top_k < a.V;
  const bool from_list = !greedy && listable(P, topk, a.V);
  // rows that may read all their elements again are finished by the whole cluster
  const bool team = ctas > 1 && !greedy && !from_list &&
                    (topk || (P.flags & (kRowTopP | kRowMinP)));
  if (rank > 0 && !team) return;
  for (int i = tid; i < kTable; i += kThreadsF) sh.table[i] = d_mass_table.v[i];
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // the row's maximum
  const float* seg_max = a.seg_max + (int64_t)row * a.segs;
  const uint64_t* seg_sum = a.seg_sum + (int64_t)row * a.segs;
  float mx = -INFINITY;
  for (int s = tid; s < a.segs; s += kThreadsF) {
    const float v = seg_max[s];
    sh.seg_max[s] = v;
    sh.seg_w[s] = seg_sum[s];
    mx = max_nan(mx, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) sh.red_f[warp] = mx;
  if (team) cluster.sync();  // every CTA of the team runs before its memory is written
  else __syncthreads();
  mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < kWarpsF; ++i) mx = max_nan(mx, sh.red_f[i]);
  const float m = __fmul_rn(mx, P.inv_t);
  const int status = isnan(mx) || m == INFINITY ? kRowNonfinite : m == -INFINITY ? kRowEmpty : kRowOk;
  int32_t* out_tok = a.out_tokens + (int64_t)row * a.draws;
  float* out_lp = a.out_logprobs ? a.out_logprobs + (int64_t)row * a.draws : nullptr;
  if (rank == 0 && tid == 0) a.row_status[row] = status;
  if (status != kRowOk) {
    if (rank == 0)
      for (int d = tid; d < a.draws; d += kThreadsF) {
        out_tok[d] = -1;
        if (out_lp) out_lp[d] = NAN;
      }
    return;
  }
  const Mass mass(P.inv_t, m, sh.table);
  const RowData<T> rd{static_cast<const T*>(a.logits) + row * a.ld, a.V, a.aligned != 0};
  Row<T> rw(rd, mass, mx, m, a.segs, a.drop, team ? ctas : 1, team ? rank : 0);

  // ln sum exp(z - m) from the segments' sums; masses to element units of the row
  float ln_s = 0.f;
  const bool masses = sums_masses(P, a.V);
  const bool usable = masses && fabsf(m) < kUsable;
  uint64_t all = 0;  // mass of every element, row units (0: not known)
  if (usable) {
    for (int s = tid; s < a.segs; s += kThreadsF) {
      const float zm = mass.z(sh.seg_max[s]);
      uint64_t w = 0;
      if (zm > -INFINITY) {
        const int sh_r = mass.E() - Mass(P.inv_t, zm, sh.table).E();
        w = fabsf(zm) < kNarrow && sh_r < 64 ? sh.seg_w[s] >> sh_r : 0;
      }
      sh.seg_w[s] = w;
      all += rw.coarse(w);
    }
    block_scan(sh, all, &all);
    ln_s = mass.ln_sum(all, kElemBits - a.drop, m);
  } else if (out_lp && !masses) {
    float e = 0.f;
    for (int s = tid; s < a.segs; s += kThreadsF) {
      const float zm = mass.z(sh.seg_max[s]);
      if (zm > -INFINITY)
        e += __uint_as_float((uint32_t)sh.seg_w[s]) *
             ex2_approx(fmaxf(fabsf(zm), fabsf(m)) < kNarrow
                            ? lse_base(zm) - lse_base(m)
                            : __fmul_rn(__fsub_rn(zm, m), kLog2e));
    }
    // lse_base(m) ln 2 - m in one rounding, ln 2 in two parts
    ln_s = logf(block_sum(sh, e)) +
           (__fmaf_rn(lse_base(m), 0.693147182464599609375f, lse_shift(m) - m) +
            lse_base(m) * -1.904654299957e-9f);
  }

  if (greedy) {
    // the lowest index at the maximum: the first segment that has it
    int first = kMaxIdx;
    for (int s = tid; s < a.segs; s += kThreadsF)
      if (sh.seg_max[s] == mx) first = min(first, s);
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.red_i[warp] = first;
    __syncthreads();
    for (int i = 0; i < kWarpsF; ++i) first = min(first, sh.red_i[i]);
    int j = kMaxIdx;
#pragma unroll 1
    for (int i = 0; i < RD::kIters; ++i) {
      float x[RD::N];
      rd.load(RD::at(first, i), x);
#pragma unroll
      for (int e = RD::N - 1; e >= 0; --e)
        if (x[e] == mx) j = min(j, RD::at(first, i) + e);
    }
    j = __reduce_min_sync(0xffffffffu, j);
    for (int d = tid; d < a.draws; d += kThreadsF) {
      out_tok[d] = j;
      if (out_lp) out_lp[d] = -ln_s;
    }
    return;
  }

  // the kept set
  Cut cut{-3.402823466e38f, kMaxIdx};
  if (P.flags & kRowMinP) {
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
  if (from_list && (!masses || usable) &&
      draw_from_list(rw, a, P, cut, topk ? P.top_k : a.V, row, ln_s))
    return;
  if (topk) {
    // (an element count decides whether top-k cuts anything)
    int c = 0;
    for (int s = rw.s0 + warp; s < rw.s1; s += kWarpsF) {
      if (rw.seg_top(s) < cut.z) continue;
#pragma unroll 1
      for (int i = 0; i < RD::kIters; ++i) {
        float x[RD::N];
        rd.load(RD::at(s, i), x);
#pragma unroll
        for (int e = 0; e < RD::N; ++e) c += rw.mass.z(x[e]) >= cut.z;
      }
    }
    rw.send(&Mail::total, block_sum(sh, c));
    rw.sync();
    int n = 0;
    for (int r = 0; r < rw.C; ++r) n += sh.mail.total[r];
    if (n > P.top_k && !band_select<T, false, true>(rw, &cut, (uint64_t)P.top_k, -INFINITY))
      cut = radix_select<T, false>(rw, cut, (uint64_t)P.top_k);
  }
  uint64_t before, mine, W;
  if (P.flags & kRowTopP) {
    if (all == 0) {  // the mass of what top-p is a share of
      kept_mass(rw, cut);
      all = sum_segments(rw, cut, &before, &mine);
      if (masses) ln_s = mass.ln_sum(all, kElemBits - a.drop, m);
    }
    const Cut from = cut;
    const uint64_t target = part_of(all, P.top_p);
    // V elements below this hold less than the share 1 - p (a logit's hundredth is
    // far more than the roundings here)
    const float z_least =
        fabsf(m) < kUsable
            ? m + (mass.ln_sum(all, kElemBits - a.drop, m) + logf((1.f - P.top_p) / (float)a.V)) -
                  0.01f
            : -INFINITY;
    bool done = false;
    if constexpr (sizeof(T) == 2) {
      if (!topk && !(P.flags & kRowMinP)) done = code_select(rw, &cut, target);
    }
    if (!done) {
      done = from.idx == kMaxIdx ? band_select<T, true, true>(rw, &cut, target, z_least)
                                 : band_select<T, true, false>(rw, &cut, target, z_least);
      if (!done) {
        cut = radix_select<T, true>(rw, from, target);
        kept_mass(rw, cut);
      }
    }
    W = sum_segments(rw, cut, &before, &mine);
  } else {
    if (!usable) kept_mass(rw, cut);
    W = sum_segments(rw, cut, &before, &mine);
    if (masses && !usable) ln_s = mass.ln_sum(W, kElemBits - a.drop, m);
  }

  // the draws: each by a warp of the CTA that holds its mass; numbers of 1 and more
  // by the last CTA with a kept element
  const bool streamed = usable && !(P.flags & kRowTopP);
  bool at_end = sh.mail.last[rw.rank] >= 0;
  for (int r = rw.rank + 1; r < rw.C; ++r) at_end = at_end && sh.mail.last[r] < 0;
  for (int d = warp; d < a.draws; d += kWarpsF) {
    const float u = a.uniforms[(int64_t)row * a.draws + d];
    float z;
    int j;
    if (u >= 1.f) {
      if (!at_end) continue;
      j = last_kept(rw, cut, sh.mail.last[rw.rank], &z);
    } else {
      const uint64_t t = part_of(W, u);
      if (t < before || t - before >= mine) continue;
      j = find_draw(rw, cut, t - before, streamed, &z);
    }
    if (lane == 0) {
      out_tok[d] = j;
      if (out_lp) out_lp[d] = __fsub_rn(__fsub_rn(z, m), ln_s);
    }
  }
}

template <typename T>
constexpr size_t stream_smem() {
  return kStreamThreads / 32 * kSeg * sizeof(T);
}

template <typename T>
cudaError_t launch_given_typed(const GivenArgs& a, int num_sms, int ctas, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.B * a.segs;
  int64_t grid = (warps + kStreamThreads / 32 - 1) / (kStreamThreads / 32);
  if (grid > (int64_t)kStreamCtas * num_sms) grid = (int64_t)kStreamCtas * num_sms;
  stream_kernel<T><<<(unsigned)grid, kStreamThreads, stream_smem<T>(), stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * ctas));
  cfg.blockDim = dim3(kThreadsF);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  // its prologue overlaps the end of stream_kernel (griddepcontrol.wait)
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, finish_kernel<T>, a);
}

}  // namespace

template <typename T>
cudaError_t prepare_given_typed() {
  cudaError_t e = cudaFuncSetAttribute(
      finish_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(stream_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)stream_smem<T>());
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(finish_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

cudaError_t prepare_given() {
  const cudaError_t e = prepare_given_typed<float>();
  return e != cudaSuccess ? e : prepare_given_typed<__nv_bfloat16>();
}

cudaError_t launch_given(GivenArgs a, int dtype, int num_sms, cudaStream_t stream) {
  a.segs = (a.V + kSeg - 1) / kSeg;
  // sums of V masses stay below 2^62
  int bits = 0;
  while ((1ll << bits) < a.V) ++bits;
  a.drop = max(kListDrop, bits + kElemBits - 62);
  // CTAs that share the rows which are read again: as many as two to an SM hold for
  // all rows, at least two (1024 fp32 rows: 491 us, with four 532; 256 bf16 rows: 127
  // and 129), and eight segments to each (5 rows of 32003: 35 us with four or
  // eight, 37 with sixteen; one row of 151936: 50 with eight, 46 with sixteen).
  // The rule counts all rows, also those whose other CTAs leave at once (greedy,
  // unfiltered and listed ones): batches of few team rows use few of the SMs.
  int ctas = 2;
  while (ctas < kMaxCtas && 2 * ctas * a.B <= 2 * num_sms && 16 * ctas <= a.segs) ctas *= 2;
  return dtype == VT_DTYPE_F32 ? launch_given_typed<float>(a, num_sms, ctas, stream)
                               : launch_given_typed<__nv_bfloat16>(a, num_sms, ctas, stream);
}

}  // namespace vt
