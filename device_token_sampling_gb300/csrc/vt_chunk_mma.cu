// vt_chunk_mma.cu -- attention of chunks on the 5th-generation tensor cores.
//
// The query rows (token, head) of a request and kv head are cut into units of up to two
// tiles of 128 rows, whole tokens each; a unit attends to the tokens up to its last row's
// position, 128 at a step.  A unit of two tiles takes every step with both; one that fits
// a tile has its steps taken by the two tiles in turn, whose results are added up at the
// end.  Two launches:
//   plan_kernel    counts what the units cost and gives every CTA its own;
//   chunk_kernel   one CTA an SM, its pieces of units one after another; units that more
//                  than one CTA worked on are put together by the last to come.
//
// Why two tiles of 128 rows: a step of 128 tokens then has 33.5 MFLOP (heads of 128) for 64
// KB of keys and values, which L2 delivers beside the products, and one tile's softmax runs
// under the other's.  Tensor memory is what limits it: one accumulator and one set of weights
// a tile and one buffer of scores for both (128 + 2 x 64 + 2 x 128 columns of 512), so that
// a unit's end and the next one's beginning do not overlap (about 6 of a tile's steps).
// Measured with 32/8 heads of 128 in bf16:
//   long chunks are bound by the tensor cores and the power cap: 4 of 2048 to 4096 tokens
//   behind up to 16384, 2.03 TFLOP in 1.2 ms, 1.68 PFLOP/s, pipe active in 80 % of the
//   cycles; one of 16384 tokens 1.76 PFLOP/s;
//   few rows over long contexts by the memory: 64 requests of 1 to 8 behind 4096 to 8192,
//   1.64 GB in 261 us, 6.3 TB/s (0.94 of a plain copy's rate);
//   small batches by latency: 4 requests of 5 tokens behind up to 600 17 us, of which the
//   plan is 3.5.
#include <type_traits>

#include "vt_paged.h"
#include "vt_umma.cuh"

namespace vt {
namespace {

constexpr int kUnitRows = 2 * kTileRows;
constexpr int kChunkThreads = 512;
constexpr int kPieces = 4;    // pieces that are known ahead
constexpr int kMasks = 8;     // steps whose token masks are kept
constexpr int kHalfStep = kTileTokens / 2;  // tokens of one product
constexpr int kWeights = kTileTokens;       // tensor memory: S, then each tile's P, then O
// warps: the softmax of each tile; then one each for the scores, the products of each
// tile, the copies of K and V of even and of odd steps, the pieces and their Q; two that
// look through V
constexpr int kScoreWarp = 8, kProductWarp = 9, kKvWarp = 11, kPieceWarp = 13, kLookWarp = 14;

// ---- the units ----------------------------------------------------------------
// Heads in one tile: a.heads of the G, a.parts times; tokens in one tile: a.tokens.  A
// virtual head is a kv head and a part of its G.
struct Request {
  int s0, n;       // its rows of q
  int before;  // tokens in front of them, none past the table's columns; below 0: the first
               // rows have no position
  int units;   // of a virtual head
};
__device__ __forceinline__ Request request(const ChunkArgs& a, int b) {
  Request r;
  const int s0 = a.starts[b], s1 = a.starts[b + 1];
  const bool fine = s0 >= 0 && s0 <= s1 && s1 <= a.T;
  r.s0 = s0;
  r.n = fine ? s1 - s0 : 0;
  r.before = min(max(a.seq_lens[b], -1) - r.n, a.cols << a.shift);
  r.units = (r.n + 2 * a.tokens - 1) / (2 * a.tokens);
  return r;
}
__device__ __forceinline__ int unit_tokens(int tokens, const Request& r, int u) {
  return min(2 * tokens, r.n - u * 2 * tokens);
}
// The end of the tokens that unit u attends to, of cap at most, and its steps (one at least,
// so that rows which attend to nothing are written).
__device__ __forceinline__ int unit_end(int tokens, int cap, const Request& r, int u) {
  return min(max(r.before + min((u + 1) * 2 * tokens, r.n), 0), cap);
}
__device__ __forceinline__ int unit_steps(int tokens, int cap, const Request& r, int u) {
  return max(1, (unit_end(tokens, cap, r, u) + kTileTokens - 1) / kTileTokens);
}
// What a step of it costs (two tiles take turns on a unit that fits one),
__device__ __forceinline__ int unit_weight(int tokens, const Request& r, int u) {
  return unit_tokens(tokens, r, u) > tokens ? 2 : 1;
}
// and what beginning and ending it costs besides.
constexpr int kUnitCost = 6;
__device__ __forceinline__ int unit_cost(int tokens, int cap, const Request& r, int u) {
  return kUnitCost + unit_steps(tokens, cap, r, u) * unit_weight(tokens, r, u);
}
__device__ __forceinline__ int unit_cost(const ChunkArgs& a, const Request& r, int u) {
  return unit_cost(a.tokens, a.cols << a.shift, r, u);
}
// floor(b / m) + floor((k + b) / m) + .. of n terms; b below 2^31, the rest below 2^24.  By
// Euclid's steps on k and m: what lies under the line, then what lies beside it.
__device__ __forceinline__ int64_t sum_of_floors(uint32_t n, uint32_t m, uint32_t k, uint32_t b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += (int64_t)(k / m) * ((int64_t)n * (n - 1) / 2) + (int64_t)n * (b / m);
    k %= m;
    b %= m;
    const uint32_t top = k * n + b;  // (k < m <= 128 from here on)
    if (top < m) break;
    n = top / m;
    b = top % m;
    const uint32_t was = m;
    m = k;
    k = was;
  }
  return sum;
}
// The cost of units u0 .. u1 - 1: a walk through a few; of more in closed form, so that a
// prompt of 10^5 tokens costs the one CTA no more than one of 1000.  (Not in line: from a
// cold cache its code's copies would cost an ordinary plan 6 us.)
constexpr int kWalk = 16;
__device__ __noinline__ int64_t many_units_cost(Request r, int tokens, int cap, int u0, int u1) {
  int64_t cost = 0;
  if (u1 == r.units) cost = unit_cost(tokens, cap, r, --u1);
  // the others have two tiles and end at before + (u + 1) k: some at nothing, some at the
  // table's end
  const int k = 2 * tokens;
  const int none = r.before < 0 ? -r.before / k : 0;
  const int some = cap < r.before ? 0 : (cap - r.before) / k;
  const int lo = min(max(none, u0), u1), hi = min(max(some, lo), u1);
  const int64_t steps =
      lo - u0 + (int64_t)(u1 - hi) * ((cap + kTileTokens - 1) / kTileTokens) +
      (hi > lo ? sum_of_floors(hi - lo, kTileTokens, k, r.before + (lo + 1) * k + kTileTokens - 1)
               : 0);
  return cost + (int64_t)kUnitCost * (u1 - u0) + 2 * steps;
}
__device__ __forceinline__ int64_t units_cost(const ChunkArgs& a, const Request& r, int u0, int u1) {
  if (u1 - u0 > kWalk) return many_units_cost(r, a.tokens, a.cols << a.shift, u0, u1);
  int64_t cost = 0;
#pragma unroll 1
  for (int u = u0; u < u1; ++u) cost += unit_cost(a, r, u);
  return cost;
}
// That of the first `count` units and heads.  The order of a request's units: the longest
// first, its heads side by side.  (So CTAs that run at the same time read the same keys and
// values from L2.)
__device__ __forceinline__ int64_t first_cost(const ChunkArgs& a, const Request& r, int64_t count) {
  const int u = r.units - (int)(count / a.heads_all), rest = (int)(count % a.heads_all);
  return a.heads_all * units_cost(a, r, u, r.units) + (rest ? (int64_t)rest * unit_cost(a, r, u - 1) : 0);
}

struct Sums2 {
  int64_t x, y;
};
constexpr int kPlanThreads = 1024;
// What a share is worth at least: a CTA more is a part more to be put together, about 1 us
// each.  5 tokens behind 12000 of one request of 20/4 heads: 44 us, shares of 1 step (all
// CTAs) 62, of 24 43; 4 requests of 5 behind 2000 32, 31 and 39.
constexpr int kLeast = 8;
constexpr int kMostRounds = 16;  // of units that are looked at one by one

// The last b with first[b] <= v.
__device__ __forceinline__ int find_request(const int64_t* first, int stride, int B, int64_t v) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[(int64_t)mid * stride] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One CTA: prefix sums of the requests' units and what they cost; then what each CTA of
// chunk_kernel does.  Units go whole, in rounds, every other round the other way about
// (a request's come longest first), or as one row of steps cut into shares:
//   - all whole, where that leaves no CTA with much more than the mean: 16 and a 16th.
//     A unit that is cut is written out in parts and put together, which costs about as
//     much as 16 steps of one tile.  us whole and cut, 32/8 heads of 128: one prompt of 1024
//     tokens 29 and 48, of 4096 107 and 129, of 8192 337 and 363; 256 requests of up to 4
//     new tokens behind up to 2000 215 and 249.  A limit of 12 left 8 prompts of 512 (54
//     and 68) cut, of 24 made 20 requests of 5 tokens behind 2000 whole (59 and 53); an 8th
//     made 4 prompts of up to 4096 whole, 9 % apart (1004 and 975).
//   - else, where some request has several units a kv head (which share keys and values)
//     and there are two rounds at least, all but the last whole round and what is behind
//     it, which goes in shares that make up for the CTAs' differences;
//   - else all in shares.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(ChunkArgs a) {
  __shared__ Sums2 s_warp[33];
  __shared__ int64_t s_first[2 * (kPlanThreads + 1)];  // plan_first, where it fits
  __shared__ int s_several, s_most;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) s_several = s_most = 0;
  __syncthreads();
  int64_t units = 0, steps = 0;
  for (int base = 0; base < a.B; base += kPlanThreads) {
    const int b = base + tid;
    int64_t x = 0, y = 0;
    if (b < a.B) {
      const Request r = request(a, b);
      const int s0 = a.starts[b], s1 = a.starts[b + 1];
      if (s0 < 0 || s0 > s1 || s1 > a.T) atomicOr(a.err_word, kErrBadRows);
      x = (int64_t)r.units * a.heads_all;
      y = units_cost(a, r, 0, r.units);
      y *= a.heads_all;
      if (r.units > 1) s_several = 1;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t px = __shfl_up_sync(0xffffffffu, x, o), py = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += px;
        y += py;
      }
    }
    __syncthreads();
    if (lane == 31) s_warp[warp + 1] = Sums2{x, y};
    __syncthreads();
    if (warp == 0) {
      int64_t vx = s_warp[lane + 1].x, vy = s_warp[lane + 1].y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t px = __shfl_up_sync(0xffffffffu, vx, o),
                      py = __shfl_up_sync(0xffffffffu, vy, o);
        if (lane >= o) {
          vx += px;
          vy += py;
        }
      }
      s_warp[lane + 1] = Sums2{vx, vy};
      if (lane == 0) s_warp[0] = Sums2{0, 0};
    }
    __syncthreads();
    x += s_warp[warp].x;
    y += s_warp[warp].y;
    if (b < a.B) {
      a.plan_first[2 * (b + 1)] = units + x;
      a.plan_first[2 * (b + 1) + 1] = steps + y;
      if (a.B <= kPlanThreads) {
        s_first[2 * (b + 1)] = units + x;
        s_first[2 * (b + 1) + 1] = steps + y;
      }
    }
    units += s_warp[32].x;
    steps += s_warp[32].y;
  }
  if (tid == 0) a.plan_first[0] = a.plan_first[1] = s_first[0] = s_first[1] = 0;
  __syncthreads();
  const int64_t* first = a.B <= kPlanThreads ? s_first : a.plan_first;
  const int G = a.grid;
  const int rounds = s_several && units >= 2 * G ? (int)units / G - 1 : 0;
  const bool maybe = units <= kMostRounds * G;
  // what the units of rounds cost, each CTA's: of all, of `rounds`
  int mine = 0;
  int64_t most = 0, want = 0;
  if (tid < G) {
    for (int i = 0; i < (maybe ? kMostRounds : rounds); ++i) {
      const int64_t u = (int64_t)i * G + (i & 1 ? G - 1 - tid : tid);
      if (u >= units) break;
      const int b = find_request(first, 2, a.B, u);
      const Request r = request(a, b);
      const int cost = unit_cost(a, r, r.units - 1 - (int)(u - first[2 * b]) / a.heads_all);
      most += cost;
      if (i < rounds) want += cost;
      ++mine;
    }
    if (maybe) atomicMax(&s_most, (int)min(most, (int64_t)0x7fffffff));
  }
  __syncthreads();
  const bool whole = maybe && (int64_t)s_most * G <= steps + steps / 16 + 16 * G;
  if (whole) {
    if (tid <= G) {
      ChunkStart s{};
      s.at = steps;  // (no share)
      s.b = a.B;
      s.rounds = mine;
      a.plan_start[tid] = s;
    }
    return;
  }
  for (int i = tid; i < 8 * G; i += kPlanThreads) a.plan_count[i] = 0;
  int64_t skipped = 0;
  if (rounds > 0) {
    const int64_t u = (int64_t)rounds * G;
    const int b = find_request(first, 2, a.B, u);
    const Request r = request(a, b);
    skipped = first[2 * b + 1] + first_cost(a, r, u - first[2 * b]);
  }
  const int64_t todo = steps - skipped;
  // The rest goes in shares that make up for it: up to the mean of all.  (Equal shares
  // left the CTAs' sums 9 % apart on 4 prompts of up to 4096 tokens.)
  // CTAs that get some
  const int some = rounds > 0 ? G : (int)min((int64_t)G, steps / kLeast + 1);
  want = tid < some ? max(steps / some + 1 - want, (int64_t)0) : 0;
  int64_t upto = want;  // of the CTAs up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 31) s_warp[warp + 1].x = upto;
  __syncthreads();
  int64_t all = 0, before = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) before += s_warp[w + 1].x;
    all += s_warp[w + 1].x;
  }
  before += upto - want;
  const int c = tid;
  if (c <= G) {
    const int64_t at = c == G ? steps : skipped + todo * before / max(all, (int64_t)1);
    ChunkStart s{};
    s.at = at;
    s.b = a.B;
    if (at < steps) {
      const int b = find_request(first + 1, 2, a.B, at);
      const Request r = request(a, b);
      int64_t left = at - first[2 * b + 1];
      int u0 = 0, u = r.units;  // the unit that it is in: from u0 on, below u
      while (u - u0 > kWalk) {
        const int mid = (u0 + u) >> 1;
        if (units_cost(a, r, mid, r.units) * a.heads_all > left) u0 = mid;
        else u = mid;
      }
      left -= units_cost(a, r, u, r.units) * a.heads_all;
      int64_t each;
      for (;;) {
        each = unit_cost(a, r, --u);
        if (u == u0 || left < each * a.heads_all) break;
        left -= each * a.heads_all;
      }
      s.b = b;
      s.unit = u;
      s.head = (int)(left / each);
      const int in = (int)(left % each), w = unit_weight(a.tokens, r, u);
      s.step = max(in - kUnitCost, 0) / w;  // (a whole step)
      s.at += (s.step > 0 ? kUnitCost + s.step * w : 0) - in;
    }
    s.rounds = rounds;
    a.plan_start[c] = s;
  }
}

// ---- what the roles of a CTA share ------------------------------------------------
template <int D>
struct ChunkSmem {
  static constexpr int kHalf = kTileRows * 128;      // 128 rows of 64 elements
  static constexpr int kTile = (D / 64) * kHalf;     // bytes of a Q, K or V tile
  static constexpr int kRing = D == 128 ? 4 : 8;     // K and V tiles
  static constexpr int kQ = 0;
  static constexpr int kKv = 2 * kTile;
  static constexpr int kRest = kKv + kRing * kTile;
};

struct Piece {
  int b, kvh, head;  // the first query head
  int heads;         // of a token here
  int token;         // the unit's first row of q
  int tokens;        // of the unit; 0: no more pieces
  int t0, t1;        // steps
  int end;           // of the unit's tokens
  int lim0;          // end of the tokens that its first row attends to
  int slot;          // of its partial result, or -1: the whole unit
  int job, last;     // a part: the CTAs that began and end the unit
  int parts;         // how many parts it has
};

template <int R>
struct Shared {
  // of the ring: what both tiles use, what one of them does (a waiter sees every use of
  // its barriers, so that a phase's parity says which it is)
  uint64_t full[2][R], empty[R];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t s_full[2], s_free;        // scores made, of each tile; read
  // of each tile, by halves of a step: weights stored; product done
  uint64_t p_full[2][2], pv_done[2][2];
  // of each tile: products of a unit done; accumulator read
  uint64_t o_done[2], o_empty[2];
  uint64_t v_ok[2][4];               // of each tile, by turns: V of a step looked through
  uint64_t x_full;                   // tile 1's sums of a unit that the tiles share, for tile 0
  uint64_t q_full[2], q_empty[2];
  uint64_t drained[4];
  float sums[2][kTileRows];         // those: maxima, sums
  Piece piece[kPieces];
  uint32_t mask[kMasks][4];
  int32_t whole[kMasks];
  uint32_t poison[4][4];             // tokens of V that are not finite, by turns
  uint32_t tmem;
};

// The ring's places: K of the CTA's step g at 2 g, V behind it, modulo R.  The tiles that
// share a unit take even and odd steps of the CTA's whole sequence, so that a place is
// always the same tile's then.
template <int R>
__device__ __forceinline__ int place(uint32_t g, int v) {
  static_assert(R == 4 || R == 8, "even and odd steps have their own places");
  return (int)((2 * g + v) & (R - 1));
}

__device__ __forceinline__ uint64_t pack_f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
// 32 columns of this thread's lane and their maximum, NaN left out
__device__ __forceinline__ void tmem_ld32_max(uint32_t (&r)[32], uint32_t& top, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : VT_R8(r, 0), VT_R8(r, 8), VT_R8(r, 16), VT_R8(r, 24), "=r"(top)
      : "r"(addr));
}
// 16 columns of this thread's lane
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : VT_R8(r, 0), VT_R8(r, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      VT_I8(r, 0), VT_I8(r, 8)
      : "memory");
}
__device__ __forceinline__ void loaded16(uint32_t (&r)[16]) {
  asm volatile("" : VT_P8(r, 0), VT_P8(r, 8)::"memory");
}
// 32 bytes, a whole sector, at once
__device__ __forceinline__ void store32(void* to, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t addr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Whether one of 8 elements is an infinity or a NaN: all exponent bits set.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(const uint4& v) {
  constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kExp = kBf ? 0x7f807f80u : 0x7c007c00u, kOne = kBf ? 0x00800080u : 0x04000400u;
  return (((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) | ((v.z & kExp) + kOne) |
          ((v.w & kExp) + kOne)) & 0x80008000u;
}

// O += P V of this thread's row for the tokens of a half that V no longer holds (bits of
// w0, w1: token tok0 + bit); O = that where it is not begun.
template <typename T, int D>
__device__ __noinline__ void add_poison(const ChunkArgs& a, const Piece& p, uint32_t w0,
                                        uint32_t w1, int tok0, int lim, bool begun, uint32_t p_at,
                                        uint32_t o_at) {
  if (!begun) {
    uint32_t o[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = 0;
    for (int c = 0; c < D; c += 32) tmem_st32(o_at + c, o);
    tmem_wait_st();
  }
  for (int q = 0; q < 2; ++q)
    for (uint32_t left = q ? w1 : w0; left; left &= left - 1) {
      const int i = q * 32 + __ffs(left) - 1, tok = tok0 + i;
      const uint32_t pair = tmem_ld1(p_at + i / 2);
      const unsigned short bits = (unsigned short)(i & 1 ? pair >> 16 : pair);
      const float weight = static_cast<float>(*reinterpret_cast<const T*>(&bits));
      const int blk = a.table[(int64_t)p.b * a.ld_table + (tok >> a.shift)];
      const T* v = static_cast<const T*>(a.v) + blk * a.block_stride +
                   (tok & ((1 << a.shift) - 1)) * a.token_stride + p.kvh * a.head_stride;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(o, o_at + c);
        tmem_wait_ld();
        loaded(o);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (tok < lim)
            o[e] = __float_as_uint(__uint_as_float(o[e]) + weight * static_cast<float>(v[c + e]));
        tmem_st32(o_at + c, o);
        tmem_wait_st();
      }
    }
}

// The 32 rows of a warp (row r0 of a unit on; this lane's goes to `row` of the output, -1:
// none) from the parts that CTAs job .. last left: their first slots but for job's second.
// Each row is rescaled to its parts' common maximum, summed and divided; the order is the
// CTAs'.  A part that holds nothing (sum 0) is not read.
template <typename T, int D>
__device__ __noinline__ void join_rows(const ChunkArgs& a, int job, int last, int r0, int64_t row) {
  constexpr int W = D / 32, kRows = 16;
  const int lane = threadIdx.x & 31;
  auto slot = [&](int k) { return (int64_t)(k == job ? 2 * job + 1 : 2 * k) * kUnitRows + r0; };
  // the CTAs from k0 on, 32 at most, that have a part: a bit each
  auto parts = [&](int k0) {
    const int k = k0 + lane;
    return __ballot_sync(0xffffffffu, k <= last && a.plan_start[k].at < a.plan_start[k + 1].at);
  };
  float m = -INFINITY, l = 0.f;
  for (int k0 = job; k0 <= last; k0 += 32)
#pragma unroll 4
    for (uint32_t left = parts(k0); left; left &= left - 1) {
      const float2 ml = row >= 0 ? __ldcg(a.part_ml + slot(k0 + __ffs(left) - 1) + lane)
                                 : make_float2(-INFINITY, 0.f);
      const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
      l = l * ex2_approx(m - base) + (ml.y == 0.f ? 0.f : ml.y * ex2_approx(ml.x - base));
      m = mn;
    }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
  for (int q = 0; q < 32; q += kRows) {
    if (!__any_sync(0xffffffffu, row >= 0 && lane >= q && lane < q + kRows)) continue;
    float acc[kRows][W] = {};
#pragma unroll 1
    for (int k0 = job; k0 <= last; k0 += 32)
#pragma unroll 1
      for (uint32_t left = parts(k0); left; left &= left - 1) {
        const int64_t at = slot(k0 + __ffs(left) - 1);
        float x[kRows][W];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const float* o = a.part_o + (at + q + i) * D + lane * W;
          if constexpr (W == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(o));
            x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(o));
            x[i][0] = v.x, x[i][1] = v.y;
          }
        }
        float f = 0.f;  // this lane's row's
        if (row >= 0) {
          const float2 ml = __ldcg(a.part_ml + at + lane);
          f = ml.y == 0.f ? 0.f : ex2_approx(ml.x - (m == -INFINITY ? 0.f : m)) * inv;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const float fi = __shfl_sync(0xffffffffu, f, q + i);
          if (fi != 0.f) {  // (a NaN too)
#pragma unroll
            for (int w = 0; w < W; ++w) acc[i][w] += x[i][w] * fi;
          }
        }
      }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t to = __shfl_sync(0xffffffffu, row, q + i);
      if (to < 0) continue;
      uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + to * D + lane * W);
#pragma unroll
      for (int w = 0; w < W / 2; ++w) out[w] = pack2<T>(acc[i][2 * w], acc[i][2 * w + 1]);
    }
  }
  if (a.lse && row >= 0) a.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

// kSmall: blocks of 1 or 2 tokens, more than 32 to a step.  (In one kernel with the others
// these lost up to 9 %.)  The copies of such blocks bound it: a prompt of 1024 tokens takes
// 80, 51, 35, 29 and 25 us in blocks of 1, 2, 4, 8 and 64.
//
// Roles of a CTA's 16 warps, each with barriers of its own towards the others: 0-3 and 4-7
// the softmax and the outputs of a tile (a row a thread, 200 registers), 8 the scores of both
// tiles by turns, 9 and 10 the products of a tile, 11 and 12 the copies of even and of odd
// steps, 13 the pieces and their Q, 14 and 15 look through V.  Every wait is bounded.
template <typename T, int D, bool kSmall>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_q) {
  using L = ChunkSmem<D>;
  constexpr int R = L::kRing;
  using Sh = Shared<R>;
  extern __shared__ __align__(1024) unsigned char dyn[];
  const uint32_t base = smem_addr(dyn);
  Sh& sh = *reinterpret_cast<Sh*>(dyn + L::kRest);
  const int tid = threadIdx.x, lane = tid & 31;
  if (base & 1023) {  // (the swizzle's atoms; no static shared memory lies in front)
    if (tid == 0) atomicOr(a.err_word, kErrInternal);
    return;
  }
  // (through a shuffle, so that the roles' control flow and addresses are known to
  // be the same in a warp: MMA operands live in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(&sh.full[0][i], 1);
      mbar_init(&sh.full[1][i], 1);
      mbar_init(&sh.empty[i], i & 1 ? 4 : 2);  // (both tiles' MMAs; V: who looks through it)
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&sh.piece_full[i], 1);
      mbar_init(&sh.piece_empty[i], 15);  // (every other warp)
    }
    for (int t = 0; t < 2; ++t) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sh.p_full[t][h], 4);
        mbar_init(&sh.pv_done[t][h], 1);
      }
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.o_done[t], 1);
      mbar_init(&sh.o_empty[t], 4);
      for (int i = 0; i < 4; ++i) mbar_init(&sh.v_ok[t][i], 2);
      mbar_init(&sh.q_full[t], 1);
      mbar_init(&sh.q_empty[t], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.drained[i], 1);
    mbar_init(&sh.s_free, 4);
    mbar_init(&sh.x_full, 4);
    fence_mbar_init();
  }
  if (warp == kScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&sh.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const long long limit = a.wait_cycles;
  bool ok = true;
  constexpr uint32_t kO = 2 * kTileTokens;

  // The next piece into `p`; false behind the last, or when the wait ran out.
  int n_piece = 0;
  auto next_piece = [&](Piece& p) {
    const int at = n_piece % kPieces;
    ok = warp_wait(&sh.piece_full[at], (n_piece / kPieces) & 1, limit);
    if (!ok) return false;
    p = sh.piece[at];
    warp_arrive(&sh.piece_empty[at]);
    ++n_piece;
    return p.tokens > 0;
  };
  // row `in` of a tile
  const int in = tid & (kTileRows - 1), in_token = in / a.heads, in_head = in % a.heads;
  const int cap = a.cols << a.shift;

  if (warp < kScoreWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax and outputs: a warpgroup to a tile, one thread to a row -----------------
    const int t = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane (warp % 4) * 32
    // (a scale of 0 as one that leaves masked scores at -inf)
    const float sc = fmaxf(fabsf(a.scale_log2), 1e-30f);
    const uint64_t sc2 = pack_f2(sc, sc);
    // this tile's steps; units, and those that the tiles share; the CTA's steps; the
    // parities of v_ok's uses
    uint32_t steps = 0, units = 0, shared = 0, all = 0, ok_ph = 0;
    Piece p;
    while (ok && next_piece(p)) {
      const bool two = p.tokens > a.tokens;  // else the tiles share the unit
      const int token = (two ? t * a.tokens : 0) + in_token;
      const bool live = token < p.tokens && in_token < a.tokens && in_head < p.heads;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const int lim = live ? min(max(p.lim0 + token, 0), cap) : 0;
      const int lim_min = __reduce_min_sync(0xffffffffu, live ? lim : 0x7fffffff);
      const int n = p.t1 - p.t0;
      float m = -INFINITY, l = 0.f;
      bool begun = false;  // (a product has been added to the accumulator)
      bool poisoned = false;
      for (int j = two ? p.t0 : p.t0 + ((all ^ t) & 1); j < p.t1 && ok;
           j += two ? 1 : 2, ++steps) {
        const uint32_t g = all + (j - p.t0);
        const int ring = g % kMasks;
        // Some row does not attend to the whole step: its weights there are 0, but 0
        // times an infinity or a NaN is NaN.
        const bool diagonal = (j + 1) * kTileTokens > max(p.lim0, 0);
        poisoned = false;
        ok = warp_wait(&sh.s_full[t], steps & 1, limit);
        if (!ok) break;
        fence_after();
        if (!warp_live) {  // (the products of these rows are never read)
          warp_arrive(&sh.s_free);
          if (diagonal) {
            ok = warp_wait(&sh.v_ok[t][g & 3], (ok_ph >> (g & 3)) & 1, limit);
            ok_ph ^= 1u << (g & 3);
          }
          for (int h = 0; h < 2 && ok; ++h) {
            if (steps > 0) ok = warp_wait(&sh.pv_done[t][h], (steps - 1) & 1, limit);
            if (ok) warp_arrive(&sh.p_full[t][h]);
          }
          continue;
        }
        uint32_t s[4][32], tops[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32_max(s[q], tops[q], tmem + lanes + q * 32);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          loaded(s[q]);
          asm volatile("" : "+r"(tops[q])::"memory");
        }
        fence_before();
        warp_arrive(&sh.s_free);
        float top = max3(fmaxf(__uint_as_float(tops[0]), __uint_as_float(tops[1])),
                         __uint_as_float(tops[2]), __uint_as_float(tops[3]));
        const int tok0 = j * kTileTokens;
        const bool flip = a.scale_log2 < 0.f;
        if (flip || !sh.whole[ring] || tok0 + kTileTokens > lim_min) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // (32 tokens that every row sees stay as they are)
            const uint32_t mask = sh.mask[ring][q];
            const int left = lim - tok0 - q * 32;
            const uint32_t keep =
                mask & (left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1);
            if (__any_sync(0xffffffffu, flip || keep != 0xffffffffu)) {
              float most = -INFINITY;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if (flip) s[q][i] ^= 0x80000000u;
                if (!((keep >> i) & 1)) s[q][i] = 0xff800000u;
                most = fmaxf(most, __uint_as_float(s[q][i]));
              }
              tops[q] = __float_as_uint(most);
            }
          }
          top = fmaxf(fmaxf(__uint_as_float(tops[0]), __uint_as_float(tops[1])),
                      fmaxf(__uint_as_float(tops[2]), __uint_as_float(tops[3])));
        }
        top *= sc;
        // The reference of the exponentials stays where it is until it is kSlack (in log2)
        // short: weights of up to 2^kSlack are rounded like the others, each relative to
        // itself, and a rescale of the accumulator is rare.
        constexpr float kSlack = 8.f;
        const bool grow = top > (m == -INFINITY ? m : m + kSlack);
        const uint32_t o_at = tmem + lanes + kO + t * D;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2_approx(m - top) : 1.f;
          if (grow) m = top;
          l *= f;
          if (begun) {
            ok = warp_wait(&sh.pv_done[t][1], (steps - 1) & 1, limit);
            if (!ok) break;
            fence_after();
            const uint64_t f2 = pack_f2(f, f);
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(o, o_at + c);
              tmem_wait_ld();
              loaded16(o);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                float x0, x1;
                unpack_f2(mul_f2(pack_f2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), f2),
                          x0, x1);
                o[i] = __float_as_uint(x0);
                o[i + 1] = __float_as_uint(x1);
              }
              tmem_st16(o_at + c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const uint64_t off2 = pack_f2(off, off);
        uint64_t sum[2] = {0, 0};
        const uint32_t p_at = tmem + lanes + kWeights + t * kHalfStep;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int e = 2 * i;
            const uint64_t z =
                fma_f2(pack_f2(__uint_as_float(s[2 * h + (e >> 5)][e & 31]),
                               __uint_as_float(s[2 * h + (e >> 5)][(e & 31) + 1])),
                       sc2, off2);
            float z0, z1;
            unpack_f2(z, z0, z1);
            const float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
            sum[i & 1] = add_f2(sum[i & 1], pack_f2(p0, p1));
            // the weights are rounded to the cache's type for the tensor cores (a
            // relative 2^-9 in bf16, 2^-12 in fp16, each its own way); the sum is not
            w[i] = pack2<T>(p0, p1);
          }
          // (the product with the last ones is done)
          if (steps > 0) ok = warp_wait(&sh.pv_done[t][h], (steps - 1) & 1, limit);
          if (!ok) break;
          fence_after();
          tmem_st32(p_at + h * 32, w);
          tmem_wait_st();
          if (diagonal) {
            if (h == 0) {
              ok = warp_wait(&sh.v_ok[t][g & 3], (ok_ph >> (g & 3)) & 1, limit);
              ok_ph ^= 1u << (g & 3);
              if (!ok) break;
              // (written again four steps on, behind a product that waits for this warp)
              const uint32_t* words = sh.poison[g & 3];
              poisoned = (words[0] | words[1] | words[2] | words[3]) != 0;
            }
            if (poisoned) {
              // what was taken out of V, for the rows that attend to it, added in front of
              // the half's product
              const bool added = begun || h > 0;
              ok = added ? warp_wait(&sh.pv_done[t][h ^ 1], (h ? steps : steps - 1) & 1, limit)
                         : warp_wait(&sh.o_empty[t], (units & 1) ^ 1, limit);
              if (!ok) break;
              fence_after();
              add_poison<T, D>(a, p, sh.poison[g & 3][h * 2], sh.poison[g & 3][h * 2 + 1],
                               tok0 + h * kHalfStep, lim, added, p_at + h * 32, o_at);
            }
          }
          fence_before();
          warp_arrive(&sh.p_full[t][h]);
        }
        begun = true;
        float s0, s1;
        unpack_f2(add_f2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      all += n;
      // (every unit's, so that a parity is the last unit's)
      ok = warp_wait(&sh.o_empty[t], (units & 1) ^ 1, limit);
      if (!ok) break;
      if (!two && t == 1) {
        sh.sums[0][in] = m;
        sh.sums[1][in] = l;
        warp_arrive(&sh.x_full);
        ++units;
        continue;
      }
      // factors of the two accumulators of a unit that the tiles share; of this tile's
      float f0 = 1.f, f1 = 0.f;
      const bool both = !two && n > 1;  // (both had steps)
      int one = t;                      // the tile of the only accumulator, or the first
      if (!two) {
        ok = warp_wait(&sh.x_full, shared & 1, limit);
        ++shared;
        if (!ok) break;
        const float m1 = sh.sums[0][in], l1 = sh.sums[1][in];
        const float mm = fmaxf(m, m1), base = mm == -INFINITY ? 0.f : mm;
        f0 = ex2_approx(m - base);
        f1 = ex2_approx(m1 - base);
        l = l * f0 + l1 * f1;
        m = mm;
        if (!both) {
          one = (all - 1) & 1;
          f0 = one ? f1 : f0;
        }
      }
      // the rows: whole ones divided by their sums, parts as they are
      const float inv = l == 0.f ? 0.f : p.slot >= 0 ? 1.f : 1.f / l;
      f0 *= inv;
      f1 *= inv;
      ok = warp_wait(&sh.o_done[t], units & 1, limit);
      if (ok && !two) ok = warp_wait(&sh.o_done[1], units & 1, limit);
      if (!ok) break;
      ++units;
      fence_after();
      const int64_t row = (int64_t)(p.token + token) * a.hq + p.head + in_head;
      const int64_t part = (int64_t)max(p.slot, 0) * kUnitRows + (two ? t * kTileRows : 0) + in;
      if (warp_live) {
        const uint32_t o_at = tmem + lanes + kO + one * D;
        T* out = static_cast<T*>(a.out) + row * D;
        float* part_o = a.part_o + part * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(o, o_at + c);
          if (both) {
            uint32_t o1[32];
            tmem_ld32(o1, o_at + D + c);
            tmem_wait_ld();
            loaded(o);
            loaded(o1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) * f0 + __uint_as_float(o1[i]) * f1);
          } else {
            tmem_wait_ld();
            loaded(o);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = f0 == 0.f ? 0u : __float_as_uint(__uint_as_float(o[i]) * f0);
          }
          if (!live) continue;
          if (p.slot >= 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) store32(part_o + c + i, &o[i]);
          } else {
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              y[i] = pack2<T>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
            if (a.out_wide) {
              store32(out + c, &y[0]);
              store32(out + c + 16, &y[8]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint4*>(out + c + 2 * i) =
                    make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
          }
        }
        fence_before();
      }
      warp_arrive(&sh.o_empty[t]);
      if (!two) warp_arrive(&sh.o_empty[1]);
      if (p.slot < 0) {
        if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
      } else if (warp_live) {
        // the last warp to leave its part of these rows puts them together
        if (live) a.part_ml[part] = make_float2(m, l);
        __threadfence();
        __syncwarp();
        int before = 0;
        if (lane == 0) before = atomicAdd(a.plan_count + p.job * 8 + (two ? t : 0) * 4 + (warp & 3), 1);
        if (__shfl_sync(0xffffffffu, before, 0) == p.parts - 1) {
          __threadfence();
          join_rows<T, D>(a, p.job, p.last, (two ? t * kTileRows : 0) + (in & ~31), live ? row : -1);
        }
      }
    }
    tmem_wait_st();  // (where a wait ran out)
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kKvWarp || warp == kKvWarp + 1) {
      // ---- keys and values of even steps, of odd steps --------------------------------------
      const int odd = warp - kKvWarp;
      const int box = min(1 << a.shift, kTileTokens);  // tokens of a copy
      const int boxes = kTileTokens / box;
      uint32_t all = 0;
      // of the full barriers: those that a copy was to complete, the parities of their
      // uses; of the places, the parities of their uses
      uint32_t used = 0, full_ph = 0, empty_ph = 0;
      Piece p;
      while (ok && next_piece(p)) {
        const int32_t* table = a.table + (int64_t)p.b * a.ld_table;
        const int set = p.tokens <= a.tokens;  // (the tiles share the unit)
        for (int j = p.t0 + ((all ^ odd) & 1); j < p.t1 && ok; j += 2) {
          const uint32_t g = all + (j - p.t0);
          const int tok0 = j * kTileTokens;
          // the blocks of this tile, up to 32 of them: one a lane
          const int tok = tok0 + lane * box;
          const bool here = lane < boxes && tok < p.end;
          int blk = here ? table[tok >> a.shift] : -1;
          const bool fine = blk >= 0 && blk < a.num_blocks;
          if (here && !fine) atomicOr(a.err_word, kErrBadBlock);
          if (!fine) blk = a.num_blocks;  // outside: the copy fills zeros
          const unsigned good = __ballot_sync(0xffffffffu, fine);
          // (the rest of them, where a block has 1 or 2 tokens)
          int more[3];
          unsigned good_more[3] = {0, 0, 0};
          if constexpr (kSmall)
            for (int i = 0; i < 3; ++i) {
              const int at = lane + 32 * (i + 1), tok = tok0 + at * box;
              const bool here = at < boxes && tok < p.end;
              more[i] = here ? table[tok >> a.shift] : -1;
              const bool fine = more[i] >= 0 && more[i] < a.num_blocks;
              if (here && !fine) atomicOr(a.err_word, kErrBadBlock);
              if (!fine) more[i] = a.num_blocks;
              good_more[i] = __ballot_sync(0xffffffffu, fine);
            }
          if (lane < 4) {
            uint32_t m = 0;
            if constexpr (kSmall) {
              if (box == 1) {
                m = lane == 0 ? good : lane == 1 ? good_more[0] : lane == 2 ? good_more[1] : good_more[2];
              } else {
                const uint32_t bits = (lane < 2 ? good : good_more[0]) >> (lane & 1) * 16;
                for (int i = 0; i < 16; ++i) m |= ((bits >> i) & 1) * 3u << 2 * i;
              }
            } else if (box >= 32) {
              m = (good >> (lane * 32 / box)) & 1 ? 0xffffffffu : 0u;
            } else {
              for (int i = 0; i < 32; i += box)
                if ((good >> ((lane * 32 + i) / box)) & 1) m |= ((1u << box) - 1) << i;
            }
            const int left = p.end - tok0 - lane * 32;
            m &= left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1;
            sh.mask[g % kMasks][lane] = m;
            const unsigned every = __ballot_sync(0xfu, m == 0xffffffffu);
            if (lane == 0) sh.whole[g % kMasks] = every == 0xfu;
          }
          __syncwarp();
          const int in_block = tok0 & ((1 << a.shift) - 1);  // (blocks longer than a tile)
          for (int kv = 0; kv < 2; ++kv) {
            const int st = place<R>(g, kv);
            ok = warp_wait(&sh.empty[st], ((empty_ph >> st) & 1) ^ 1, limit);
            if (!ok) break;
            empty_ph ^= 1u << st;
            const uint32_t bit = 1u << (set * R + st);
            used |= bit;
            full_ph ^= bit;
            uint64_t* bar = &sh.full[set][st];
            if (lane == 0) mbar_arrive_expect_tx(bar, L::kTile);
            __syncwarp();
            // (the swizzle goes by the address, so that parts of its atoms of 8 tokens may come
            // from copies of their own)
            if (lane < boxes)
              for (int h = 0; h < D / 64; ++h)
                tma_tile(base + L::kKv + st * L::kTile + h * L::kHalf + lane * box * 128,
                         kv ? &map_v : &map_k, bar, h * 64, in_block, p.kvh, blk);
            if constexpr (kSmall)
              for (int i = 0; i < 3; ++i)
                if (lane + 32 * (i + 1) < boxes)
                  for (int h = 0; h < D / 64; ++h)
                    tma_tile(base + L::kKv + st * L::kTile + h * L::kHalf +
                                 (lane + 32 * (i + 1)) * box * 128,
                             kv ? &map_v : &map_k, bar, h * 64, in_block, p.kvh, more[i]);
          }
        }
        all += p.t1 - p.t0;
      }
      // no copy is in flight when the CTA's memory goes to another
      for (int i = 0; i < 2 * R; ++i)  // (the last use of each)
        if ((used >> i) & 1)
          mbar_wait_clocked(&sh.full[i / R][i % R], ((full_ph >> i) & 1) ^ 1, kDrainCycles);
    } else if (warp == kPieceWarp) {
      // ---- the pieces, and their rows of Q -------------------------------------------------
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const int G = a.grid, c = blockIdx.x;
      const ChunkStart s0 = a.plan_start[c];
      const int64_t stop = a.plan_start[c + 1].at;
      int64_t at = s0.at;
      int b = s0.b, unit = s0.unit, head = s0.head, step = s0.step;
      uint32_t uses[2] = {0, 0};
      int round = 0;
      for (int k = 0; ok; ++k) {
        Piece p{};
        const bool whole = round < s0.rounds;
        if (whole || at < stop) {
          int pb = b, pu = unit, ph = head;
          if (whole) {  // every other round the other way about
            const int64_t u = (int64_t)round * G + (round & 1 ? G - 1 - c : c);
            ++round;
            pb = find_request(a.plan_first, 2, a.B, u);
            const int i = (int)(u - a.plan_first[2 * pb]);
            ph = i % a.heads_all;
            pu = i / a.heads_all;  // (from the last)
          }
          const Request r = request(a, pb);
          if (whole) pu = r.units - 1 - pu;
          const int n = unit_steps(a.tokens, cap, r, pu);
          p.b = pb;
          p.kvh = ph / a.parts;
          const int part = ph % a.parts * a.heads;
          p.head = p.kvh * a.G + part;
          p.heads = min(a.heads, a.G - part);
          p.token = r.s0 + pu * 2 * a.tokens;
          p.tokens = unit_tokens(a.tokens, r, pu);
          p.end = unit_end(a.tokens, cap, r, pu);
          p.lim0 = r.before + pu * 2 * a.tokens + 1;
          p.t0 = 0;
          p.t1 = n;
          p.slot = -1;
          if (!whole) {  // the rest of a unit, or of this CTA's share
            const int w = unit_weight(a.tokens, r, pu);
            const int64_t begin = at - (step > 0 ? kUnitCost + (int64_t)step * w : 0);
            const int64_t end = begin + kUnitCost + (int64_t)n * w;
            p.t0 = step;
            p.t1 = stop >= end ? n : (int)((stop - begin - kUnitCost) / w);
            p.slot = step > 0 ? 2 * c : p.t1 < n ? 2 * c + 1 : -1;
            if (p.slot >= 0) {  // who else has some of the unit
              p.job = c;
              while (p.job > 0 && a.plan_start[p.job].at > begin) --p.job;
              p.last = c;
              while (p.last + 1 < G && a.plan_start[p.last + 1].at < end) ++p.last;
              for (int q = p.job; q <= p.last; ++q)
                p.parts += a.plan_start[q].at < a.plan_start[q + 1].at;
            }
            at = min(end, stop);
            step = 0;
            if (++head == a.heads_all) {
              head = 0;
              if (--unit < 0 && at < stop) {
                do ++b;
                while (b < a.B - 1 && request(a, b).units == 0);
                unit = request(a, b).units - 1;
              }
            }
          }
        }
        ok = warp_wait(&sh.piece_empty[k % kPieces], ((k / kPieces) & 1) ^ 1, limit);
        if (!ok) break;
        if (lane == 0) sh.piece[k % kPieces] = p;
        warp_arrive(&sh.piece_full[k % kPieces]);
        if (p.tokens == 0) break;
        // (rows that are not this unit's are never used)
        for (int t = 0; t < 2 && ok; ++t) {
          ok = warp_wait(&sh.q_empty[t], (uses[t] & 1) ^ 1, limit);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sh.q_full[t], a.q_bytes);
            for (int h = 0; h < D / 64; ++h)
              tma_tile(base + L::kQ + t * L::kTile + h * L::kHalf, &map_q, &sh.q_full[t], h * 64,
                       p.head - p.kvh * a.G, p.kvh,
                       p.token + (p.tokens > a.tokens ? t * a.tokens : 0));
          }
          __syncwarp();
          ++uses[t];
        }
      }
      // no copy is in flight when the CTA's memory goes to another
      for (int t = 0; t < 2; ++t)
        if (uses[t] > 0) mbar_wait_clocked(&sh.q_full[t], (uses[t] - 1) & 1, kDrainCycles);
    } else if (warp >= kLookWarp) {
      // ---- V of the steps that some row does not attend to the whole of -----------------------
      // Its weights there are 0, but 0 times an infinity or a NaN is NaN: tokens that are
      // not finite are taken out.  64 tokens to a warp, two to a lane.
      const int mine = warp - kLookWarp;
      uint32_t all = 0, full_ph[2] = {0, 0};
      Piece p;
      while (ok && next_piece(p)) {
        const bool two = p.tokens > a.tokens;
        uint32_t ph = two ? full_ph[0] : full_ph[1];
        for (int j = p.t0; j < p.t1 && ok; ++j, ++all) {
          const int st = place<R>(all, 1);
          ok = warp_wait(&sh.full[!two][st], (ph >> st) & 1, limit);
          ph ^= 1u << st;
          if (!ok) break;
          if ((j + 1) * kTileTokens > max(p.lim0, 0)) {
            bool found = false;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
              const int token = (mine * 2 + q) * 32 + lane;
              uint4* row = reinterpret_cast<uint4*>(dyn + L::kKv + st * L::kTile + token * 128);
              uint32_t bad = 0;
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  bad |= not_finite<T>(row[h * (L::kHalf / 16) + ((i + lane) & 7)]);
              if (bad) {
                found = true;
#pragma unroll 1
                for (int h = 0; h < D / 64; ++h)
                  for (int i = 0; i < 8; ++i) row[h * (L::kHalf / 16) + i] = make_uint4(0, 0, 0, 0);
              }
              const uint32_t word = __ballot_sync(0xffffffffu, bad && j * kTileTokens + token < p.end);
              if (lane == 0) sh.poison[all & 3][mine * 2 + q] = word;
            }
            if (found) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            const int from = two ? 0 : all & 1, to = two ? 2 : from + 1;
            for (int t = from; t < to; ++t) warp_arrive(&sh.v_ok[t][all & 3]);
          }
          warp_arrive(&sh.empty[st]);
        }
        if (two) full_ph[0] = ph;
        else full_ph[1] = ph;
      }
    } else if (warp < kKvWarp) {
      // ---- MMAs: a warp to the scores of both tiles by turns, one to each tile's products,
      // walk the steps and wait; one lane issues
      constexpr uint32_t kType = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      // fp32 accumulators; K-major A and B; N = 128 tokens, M = 128
      constexpr uint32_t kIdescS = (1u << 4) | (kType << 7) | (kType << 10) |
                                   ((kTileTokens / 8) << 17) | ((kTileRows / 16) << 24);
      // B (V) is N-major: its rows are tokens; N = D
      constexpr uint32_t kIdescO = (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) |
                                   ((uint32_t)(D / 8) << 17) | ((kTileRows / 16) << 24);
      constexpr uint32_t kHi = desc_hi(1024);
      // units; the CTA's steps; of the ring's places by set, the parities of their uses
      uint32_t units = 0, all = 0, full_ph[2] = {0, 0};
      Piece p;
      if (warp == kScoreWarp) {
        const uint32_t q_lo = desc_lo(base + L::kQ, 16), k_lo = desc_lo(base + L::kKv, 16);
        uint32_t scores = 0;  // of both tiles
        while (ok && next_piece(p)) {
          const bool two = p.tokens > a.tokens;
          const int n = p.t1 - p.t0;
          uint32_t ph = two ? full_ph[0] : full_ph[1];
          for (int t = 0; t < 2 && ok; ++t) ok = warp_wait(&sh.q_full[t], units & 1, limit);
          if (ok && !two && n == 1) warp_arrive(&sh.q_empty[(all & 1) ^ 1]);
#pragma unroll 1
          for (int j = 0; j < n && ok; ++j) {
            const int st = place<R>(all + j, 0);
            ok = warp_wait(&sh.full[!two][st], (ph >> st) & 1, limit);
            ph ^= 1u << st;
            const int from = two ? 0 : (all + j) & 1, to = two ? 2 : from + 1;
#pragma unroll 1
            for (int t = from; t < to; ++t, ++scores) {  // S = Q K^T
              // the last scores have been read
              if (ok && scores > 0) ok = warp_wait(&sh.s_free, (scores - 1) & 1, limit);
              if (!ok) break;
              fence_after();
              if (elect_one()) {
                const uint32_t a_lo = q_lo + t * (L::kTile >> 4), b_lo = k_lo + st * (L::kTile >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                  const uint32_t off = ((ks / 4) * L::kHalf + (ks % 4) * 32) >> 4;
                  mma_ss(tmem, a_lo + off, b_lo + off, kHi, kIdescS, ks > 0);
                }
                mma_commit(&sh.s_full[t]);
                mma_commit(&sh.empty[st]);
                if (!two) mma_commit(&sh.empty[st]);
                if (j + (two ? 1 : 2) >= n) mma_commit(&sh.q_empty[t]);
              }
              __syncwarp();
            }
          }
          if (two) full_ph[0] = ph;
          else full_ph[1] = ph;
          all += n;
          ++units;
        }
      } else {
        const int t = warp - kProductWarp;
        const uint32_t v_lo = desc_lo(base + L::kKv, L::kHalf);
        const uint32_t p_at = tmem + kWeights + t * kHalfStep, o_at = tmem + kO + t * D;
        uint32_t steps = 0;  // of this tile
        while (ok && next_piece(p)) {
          const bool two = p.tokens > a.tokens;
          const int first = two ? 0 : (all ^ t) & 1, by = two ? 1 : 2, n = p.t1 - p.t0;
          uint32_t ph = two ? full_ph[0] : full_ph[1];
          // (every unit's waits and arrivals, so that a parity is the last unit's)
          ok = warp_wait(&sh.o_empty[t], (units & 1) ^ 1, limit);
          if (ok && first >= n) warp_arrive(&sh.o_done[t]);
#pragma unroll 1
          for (int j = first; j < n && ok; j += by, ++steps) {
            const int st = place<R>(all + j, 1);
            ok = warp_wait(&sh.full[!two][st], (ph >> st) & 1, limit);
            ph ^= 1u << st;
            if (!ok) break;
            bool poisoned = false;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {  // O += P V
              ok = warp_wait(&sh.p_full[t][h], steps & 1, limit);
              if (!ok) break;
              if (j == first && (p.t0 + j + 1) * kTileTokens > max(p.lim0, 0)) {
                const uint32_t* words = sh.poison[(all + j) & 3];
                poisoned = (words[0] | words[1] | words[2] | words[3]) != 0;
              }
              fence_after();
              if (elect_one()) {
                const uint32_t b_lo = v_lo + st * (L::kTile >> 4) + h * (kHalfStep * 128 >> 4);
#pragma unroll
                for (int ks = 0; ks < kHalfStep / 16; ++ks)
                  mma_ts(o_at, p_at + h * 32 + ks * 8, b_lo + (ks * 16 * 128 >> 4), kHi, kIdescO,
                         ks > 0 ? 1u : (uint32_t)(j > first || h > 0 || poisoned));
                mma_commit(&sh.pv_done[t][h]);
                if (h) {
                  mma_commit(&sh.empty[st]);
                  if (!two) mma_commit(&sh.empty[st]);
                  if (j + by >= n) mma_commit(&sh.o_done[t]);
                }
              }
              __syncwarp();
            }
          }
          if (two) full_ph[0] = ph;
          else full_ph[1] = ph;
          all += n;
          ++units;
        }
      }
      // none of its MMAs is in flight when the CTA's memory goes to another
      uint64_t* drained = &sh.drained[warp - kScoreWarp];
      if (elect_one()) mma_commit(drained);
      __syncwarp();
      mbar_wait_clocked(drained, 0, kDrainCycles);
    }
  }
  if (!ok) atomicOr(a.err_word, kErrTimeout);
  fence_before();
  __syncthreads();
  if (warp == kScoreWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D>
constexpr size_t chunk_smem() {
  return ChunkSmem<D>::kRest + sizeof(Shared<ChunkSmem<D>::kRing>);
}
static_assert(chunk_smem<128>() <= 232448, "227 KB to a CTA");

template <typename T, int D>
cudaError_t launch_typed(const ChunkArgs& a, const CUtensorMap& mk, const CUtensorMap& mv,
                         const CUtensorMap& mq, cudaStream_t stream) {
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)a.grid);
  cfg.blockDim = dim3(kChunkThreads);
  cfg.dynamicSmemBytes = chunk_smem<D>();
  return a.shift < 2 ? cudaLaunchKernelEx(&cfg, chunk_kernel<T, D, true>, a, mk, mv, mq)
                     : cudaLaunchKernelEx(&cfg, chunk_kernel<T, D, false>, a, mk, mv, mq);
}

template <typename T, int D, bool kSmall>
cudaError_t prepare_kernel() {
  // the roles divide up 128 registers a thread: with fewer at launch they would wait
  // for the rest
  cudaFuncAttributes is;
  const cudaError_t e = cudaFuncGetAttributes(&is, chunk_kernel<T, D, kSmall>);
  if (e != cudaSuccess) return e;
  if (is.numRegs != 128) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(chunk_kernel<T, D, kSmall>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)chunk_smem<D>());
}
template <typename T, int D>
cudaError_t prepare_typed() {
  const cudaError_t e = prepare_kernel<T, D, false>();
  return e != cudaSuccess ? e : prepare_kernel<T, D, true>();
}

}  // namespace

cudaError_t prepare_chunk() {
  cudaError_t e;
  if ((e = prepare_typed<__nv_bfloat16, 64>()) || (e = prepare_typed<__nv_bfloat16, 128>()) ||
      (e = prepare_typed<__half, 64>()) || (e = prepare_typed<__half, 128>()))
    return e;
  encode_tiled();  // the driver's entry point, looked up once
  return cudaSuccess;
}

int64_t chunk_part_rows(int grid) { return 2ll * grid * kUnitRows; }

bool chunk_mma_takes(const ChunkArgs& a) {
  const int64_t most = 1ll << 38;
  return cache_map_takes(a.block_stride, a.token_stride, a.head_stride) && a.q_row > 0 &&
         a.q_head > 0 && a.q_row < most && a.q_head * a.G < most;
}

// q as [row][kv head][head][element], a tile of a.tokens rows and a.heads heads at a time.
static bool q_map(CUtensorMap* map, const ChunkArgs& a, int dtype, int head_dim) {
  const cuuint64_t dims[4] = {(cuuint64_t)head_dim, (cuuint64_t)a.G, (cuuint64_t)a.hkv,
                              (cuuint64_t)a.T};
  const cuuint64_t strides[3] = {(cuuint64_t)a.q_head * 2, (cuuint64_t)a.q_head * a.G * 2,
                                 (cuuint64_t)a.q_row * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)a.heads, 1, (cuuint32_t)a.tokens};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return encode_tiled()(map,
                        dtype == VT_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        4, const_cast<void*>(a.q), dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_chunk_mma(ChunkArgs a, int dtype, int head_dim, cudaStream_t stream) {
  // whole tokens of a kv head's G query heads to a tile of 128 rows (G = 7: 18 tokens, 126
  // rows); more heads than rows in equal parts
  a.parts = (a.G + kTileRows - 1) / kTileRows;
  a.heads = (a.G + a.parts - 1) / a.parts;
  a.tokens = kTileRows / a.heads;
  a.heads_all = a.hkv * a.parts;
  a.q_bytes = (uint32_t)(a.heads * a.tokens * head_dim * 2);
  a.out_wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  CUtensorMap mk, mv, mq;
  if (!cache_map(&mk, a.k, dtype, head_dim, a.shift, a.hkv, a.num_blocks, a.block_stride,
                 a.token_stride, a.head_stride) ||
      !cache_map(&mv, a.v, dtype, head_dim, a.shift, a.hkv, a.num_blocks, a.block_stride,
                 a.token_stride, a.head_stride) ||
      !q_map(&mq, a, dtype, head_dim))
    return cudaErrorInvalidValue;
  if (dtype == VT_DTYPE_BF16)
    return head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(a, mk, mv, mq, stream)
                           : launch_typed<__nv_bfloat16, 64>(a, mk, mv, mq, stream);
  return head_dim == 128 ? launch_typed<__half, 128>(a, mk, mv, mq, stream)
                         : launch_typed<__half, 64>(a, mk, mv, mq, stream);
}

}  // namespace vt
