// vt_tables.cu -- block tables and slot maps from request lengths.
//
// For request r with len_r tokens in blocks of 2^shift:
//   blocks_r = ceil(len_r / 2^shift), shared_r = min(blocks_r, prefix blocks),
//   have_r = max(held_r, shared_r), need_r = max(0, blocks_r - have_r),
//   off_r = the needs of the requests before r that got their blocks;
//   table[r][held_r..shared_r) = prefix blocks,
//   table[r][have_r + i] = free[cursor + off_r + i], i < need_r;
// and the token at position p of r lives in slot table[r][p >> shift] <<
// shift | (p mod 2^shift).  A request whose blocks do not fit what is left of the
// free list, or whose lengths are not valid, gets none and uses none.  Where all fit,
// off is one prefix sum.  Else the sum is taken again behind the first request that
// does not fit, without those that want more than is left (what is left only
// shrinks): once for each request that is refused because of the others in its 512.
//
// One launch, in which no CTA waits for another: every CTA scans all B
// requests itself (12 bytes a request, from L2), keeps the two prefix sums in
// shared memory and then writes its own part of the table and of the slot map.
// A token's block is worked out from its source (old table entry, prefix or
// free list), never read from an entry that this launch writes.  What bounds it:
// launch latency for a decode step's sizes (5.5 us), its instructions for prompts
// (2048 requests of up to 8192 tokens, 16.7 M places in blocks of 16: 47 us, 207 MB
// at 4.4 TB/s; 68 instructions to a lane's place, issued in 72 % of the cycles; a
// warp to a stretch of up to 512 tokens; 56 us with four tokens to a thread, which
// finds its request for every four).
#include "vt_device.cuh"
#include "vt_paged.h"
#include "vt_sampler.h"

namespace vt {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kMaxShare = 512;  // tokens of the slot map a warp takes at a time
constexpr int kColsPerItem = 256;

struct RowNeed {
  int64_t need, query;
  int held, have, blocks;
  bool bad;
};

__device__ __forceinline__ RowNeed row_need(const TablesArgs& a, int r) {
  RowNeed n;
  const int64_t len = a.seq_lens[r], q = a.query_lens[r];
  const int64_t blocks = (len + (1ll << a.shift) - 1) >> a.shift;
  n.bad = len < 0 || q < 0 || q > len || blocks > a.cols;
  n.blocks = n.bad ? 0 : (int)blocks;
  const int h = a.held ? a.held[r] : 0;
  n.held = min(max(h, 0), a.cols);
  n.have = max(n.held, min(n.blocks, a.n_prefix));
  n.need = n.bad ? 0 : max(0, n.blocks - n.have);
  n.query = n.bad ? 0 : q;
  return n;
}

struct Sums {  // needed blocks, new tokens
  int64_t x, y;
};
__device__ __forceinline__ void warp_scan2(int64_t& x, int64_t& y) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t px = __shfl_up_sync(0xffffffffu, x, o), py = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += px;
      y += py;
    }
  }
}
// Inclusive block scan of two values; s[kTabWarps] gets the totals.  The warps'
// sums are added up by warp 0 (by every thread for itself: 7 us more for 2048
// requests in 608 CTAs).
__device__ __forceinline__ void block_scan2(int64_t& x, int64_t& y, Sums* s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  __syncthreads();
  warp_scan2(x, y);
  if (lane == 31) s[w + 1] = Sums{x, y};
  __syncthreads();
  if (w == 0) {
    Sums v = lane > 0 && lane <= kTabWarps ? s[lane] : Sums{0, 0};
    warp_scan2(v.x, v.y);
    if (lane <= kTabWarps) s[lane] = v;
  }
  __syncthreads();
  x += s[w].x;
  y += s[w].y;
}

__device__ __forceinline__ int clamp31(int64_t v) {
  return (int)(v > 0x7fffffffll ? 0x7fffffffll : v);
}

__global__ void __launch_bounds__(kTabThreads, 4) tables_kernel(TablesArgs a) {
  extern __shared__ int32_t dyn[];
  int32_t* s_start = dyn;             // [B + 1] first token of each request
  int32_t* s_off = dyn + a.B + 1;     // [B] first free-list entry, or -1: the request got none
  __shared__ Sums sums[kTabWarps + 1];
  __shared__ int s_stop;
  __shared__ int64_t s_before;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first = blockIdx.x == 0;
  const int c_in = a.cursor[0];
  const int64_t c0 = c_in < 0 ? a.n_free : min(c_in, a.n_free);  // outside: nothing is free
  int64_t left = a.n_free - c0;  // of the free list, behind the requests so far
  int64_t tokens = 0;
  for (int base = 0; base < a.B; base += kTabThreads) {
    const int r = base + tid;
    RowNeed n{};
    if (r < a.B) n = row_need(a, r);
    int64_t off = -1;  // first free-list entry
    bool open = true;  // neither admitted nor refused
    bool sum_tokens = true;
    for (;;) {
      const bool fits = open && n.need <= left;
      int64_t x = fits ? n.need : 0, y = sum_tokens ? n.query : 0;
      if (tid == 0) s_stop = kTabThreads;
      block_scan2(x, y, sums);
      const int64_t want = sums[kTabWarps].x;
      if (sum_tokens && r < a.B) {
        s_start[r + 1] = clamp31(tokens + y);
        if (first) a.starts[r + 1] = clamp31(tokens + y);
      }
      tokens += sums[kTabWarps].y;
      sum_tokens = false;
      const int64_t at = a.n_free - left + x - n.need;
      if (want <= left) {
        if (fits) off = at;
        left -= want;
        break;
      }
      // the first that does not fit behind the others; those before it are settled
      if (fits && x > left) atomicMin(&s_stop, tid);
      __syncthreads();
      const int stop = s_stop;
      if (fits && tid < stop) off = at;
      if (tid == stop) s_before = x - n.need;
      open = open && tid > stop;
      __syncthreads();
      left -= s_before;
    }
    if (r < a.B) {
      const bool full = off < 0;
      const bool ok = !n.bad && !full;
      s_off[r] = ok ? clamp31(off) : -1;
      if (first) {
        a.out_held[r] = ok ? max(n.held, n.blocks) : n.held;
        a.status[r] = n.bad ? 2 : full ? 1 : 0;
      }
    }
  }
  if (tid == 0) {
    s_start[0] = 0;
    if (first) {
      a.starts[0] = 0;
      const int64_t end = a.n_free - left;
      a.out_cursor[0] = end > c0 ? (int)end : c_in;
    }
  }
  __syncthreads();

  // the table: (request, 256 columns) items over the warps of the grid
  const int per_row = (a.cols + kColsPerItem - 1) / kColsPerItem;
  const int64_t items = (int64_t)a.B * per_row;
  for (int64_t it = (int64_t)blockIdx.x * kTabWarps + warp; it < items;
       it += (int64_t)gridDim.x * kTabWarps) {
    const int r = (int)(it / per_row);
    const int c_lo = (int)(it % per_row) * kColsPerItem;
    const int c_hi = min(a.cols, c_lo + kColsPerItem);
    const RowNeed n = row_need(a, r);
    const int off = s_off[r];
    const int live = off >= 0 ? n.blocks : 0;
    const int from = max(c_lo, n.held), to = a.held ? min(c_hi, live) : c_hi;
    int32_t* row = a.table + (int64_t)r * a.ld;
    for (int c = from + lane; c < to; c += 32) {
      int id = -1;
      if (c < live) id = c < n.have ? a.prefix[c] : a.free_blocks[off + (c - n.have)];
      row[c] = id;
    }
  }

  // the slot map: a warp takes `share` tokens in a row, two neighbours a lane at a
  // time; a lane looks its request up once and walks on from there
  const int total = s_start[a.B];
  for (int64_t base = ((int64_t)blockIdx.x * kTabWarps + warp) * a.share; base < a.capacity;
       base += (int64_t)gridDim.x * kTabWarps * a.share) {
    int r = -1, r_end = 0, off = -1, shift_pos = 0;
    RowNeed n{};
#pragma unroll 1
    for (int i = 0; i < a.share; i += 64) {
      const int64_t t0 = base + i + lane * 2;
      if (t0 >= a.capacity) break;
      longlong2 slot = make_longlong2(-1, -1);
      int2 pos = make_int2(-1, -1);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t t64 = t0 + e;
        if (t64 >= total) break;
        const int t = (int)t64;
        if (r < 0 || t >= r_end) {
          if (r < 0) {  // the last request that starts at or before t: it holds t
            int lo = 0, hi = a.B;
            while (hi - lo > 1) {
              const int mid = (lo + hi) >> 1;
              if (s_start[mid] <= t) lo = mid;
              else hi = mid;
            }
            r = lo;
          } else {
            do ++r;
            while (t >= s_start[r + 1]);
          }
          r_end = s_start[r + 1];
          n = row_need(a, r);
          off = s_off[r];
          shift_pos = (int)(a.seq_lens[r] - n.query) - s_start[r];
        }
        if (off < 0) continue;
        const int p = t + shift_pos, c = p >> a.shift;
        const int id = c < n.held   ? a.table[(int64_t)r * a.ld + c]
                       : c < n.have ? a.prefix[c]
                                    : a.free_blocks[off + (c - n.have)];
        const int64_t at = ((int64_t)id << a.shift) + (p & ((1 << a.shift) - 1));
        if (e == 0) {
          pos.x = p;
          slot.x = at;
        } else {
          pos.y = p;
          slot.y = at;
        }
      }
      if (a.vec && t0 + 1 < a.capacity) {
        *reinterpret_cast<longlong2*>(a.slots + t0) = slot;
        *reinterpret_cast<int2*>(a.positions + t0) = pos;
      } else {
        a.slots[t0] = slot.x;
        a.positions[t0] = pos.x;
        if (t0 + 1 < a.capacity) {
          a.slots[t0 + 1] = slot.y;
          a.positions[t0 + 1] = pos.y;
        }
      }
    }
  }
}

}  // namespace

cudaError_t prepare_tables() {
  return cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(int32_t) * (2 * VT_PAGED_MAX_BATCH + 1));
}

cudaError_t launch_tables(TablesArgs a, int num_sms, cudaStream_t stream) {
  const size_t smem = sizeof(int32_t) * (2 * (size_t)a.B + 1);
  // shares so small that four CTAs an SM have one each, if the map is not longer
  const int64_t most = 4 * num_sms;
  const int64_t fill = (a.capacity + most * kTabWarps - 1) / (most * kTabWarps);
  a.share = (int32_t)((fill < kMaxShare ? fill + 63 : kMaxShare) / 64 * 64);
  if (a.share < 64) a.share = 64;
  const int64_t tiles = (a.capacity + kTabWarps * a.share - 1) / (kTabWarps * a.share);
  const int64_t items =
      ((int64_t)a.B * ((a.cols + kColsPerItem - 1) / kColsPerItem) + 4 * kTabWarps - 1) /
      (4 * kTabWarps);
  int64_t grid = tiles > items ? tiles : items;
  if (grid > most) grid = most;
  if (grid < 1) grid = 1;
  tables_kernel<<<(unsigned)grid, kTabThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace vt
