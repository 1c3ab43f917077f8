// vt_blocks.cu -- the life of cache blocks behind the step that took them off the
// free list: rows that continue other rows (fork), blocks that no row holds any more
// (release), blocks in use moved to the low ids (compact), and the copies that these
// ask for.
//
// Which blocks are in use is not counted along the way: it is what the rows of the
// table and the shared prefix name, one bit a block, made anew by each release or
// compact.  So a block that several rows share needs no count of its holders.
#include "vt_device.cuh"
#include "vt_paged.h"
#include "vt_sampler.h"

namespace vt {
namespace {

constexpr int kBlkThreads = 512;
constexpr int kBlkWarps = kBlkThreads / 32;
constexpr int kBlkCols = 256;  // columns of a table row a warp takes at a time

__device__ __forceinline__ int warp_scan_i(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}
// Inclusive sums over the block; *total gets that of all.  s: kBlkWarps + 1.
__device__ __forceinline__ int block_scan_i(int v, int* s, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  v = warp_scan_i(v);
  __syncthreads();
  if (lane == 31) s[w] = v;
  __syncthreads();
  if (w == 0) {
    int x = lane < kBlkWarps ? s[lane] : 0;
    x = warp_scan_i(x);
    if (lane < kBlkWarps) s[lane] = x;
  }
  __syncthreads();
  *total = s[kBlkWarps - 1];
  return v + (w > 0 ? s[w - 1] : 0);
}

// ---- fork --------------------------------------------------------------------
// Row r of the new table continues row p = parents[r] of the old one.  The lowest r of
// a parent keeps its row as it is.  The others share its blocks as far as its tokens
// reach, ceil(len / 2^shift) of them; a last one that is not full, which both will
// write into, becomes a new block off the free list and a copy.
//
// Every CTA goes through all rows itself (as the tables' kernel does) and then writes
// its own part of the table, so that one launch is enough: 512
// rows of 160 columns from 128 take 5.5 us, which is latency.
constexpr int kNoBlock = -1, kRefused = -2, kInvalid = -3;  // s_new, else the free list's index

__global__ void __launch_bounds__(kBlkThreads) fork_kernel(ForkArgs a) {
  extern __shared__ int32_t dyn[];
  int32_t* s_first = dyn;        // [B] the lowest row of each parent
  int32_t* s_new = dyn + a.B;    // [R]
  __shared__ int s_scan[kBlkWarps + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool head = blockIdx.x == 0;
  for (int i = tid; i < a.B; i += kBlkThreads) s_first[i] = 0x7fffffff;
  __syncthreads();
  for (int r = tid; r < a.R; r += kBlkThreads) {
    const int p = a.parents[r];
    if (p >= 0 && p < a.B) atomicMin(&s_first[p], r);
  }
  __syncthreads();
  const int c_in = a.cursor[0];
  const int c0 = c_in < 0 || c_in > a.n_free ? a.n_free : c_in;  // outside: nothing is free
  int taken = 0;
  for (int base = 0; base < a.R; base += kBlkThreads) {
    const int r = base + tid;
    int p = -1, len = 0, held = 0, blocks = 0, kind = kNoBlock;
    bool need = false, stays = false;
    if (r < a.R) {
      p = a.parents[r];
      if (p >= 0 && p < a.B) {
        len = a.seq_lens[p];
        held = a.held[p];
        blocks = (int)(((int64_t)len + (1 << a.shift) - 1) >> a.shift);
        if (len < 0 || held < 0 || held > a.cols || blocks > held) kind = kInvalid;
        stays = s_first[p] == r;
        need = kind != kInvalid && !stays && (len & ((1 << a.shift) - 1)) != 0;
      } else if (p != -1) {
        kind = kInvalid;
      }
    }
    int total;
    const int rank = taken + block_scan_i(need, s_scan, &total) - 1;
    taken += total;
    int id = -1;
    if (need) {
      const bool fits = rank < a.n_free - c0;
      kind = fits ? c0 + rank : kRefused;
      if (fits) id = a.free_blocks[c0 + rank];
    }
    if (r < a.R) {
      s_new[r] = kind;
      if (head) {
        const bool ok = kind >= kNoBlock && p >= 0;
        a.out_held[r] = !ok ? 0 : stays ? held : blocks;
        a.out_seq[r] = ok ? len : 0;
        a.src[r] = id >= 0 ? a.table[(int64_t)p * a.ld + blocks - 1] : -1;
        a.dst[r] = id;
        a.status[r] = kind == kInvalid ? 2 : kind == kRefused ? 1 : 0;
      }
    }
  }
  if (head && tid == 0) {
    const int got = min(taken, a.n_free - c0);
    a.out_cursor[0] = got > 0 ? c0 + got : c_in;
  }
  __syncthreads();

  const int per_row = (a.cols + kBlkCols - 1) / kBlkCols;
  const int64_t items = (int64_t)a.R * per_row;
  for (int64_t it = (int64_t)blockIdx.x * kBlkWarps + warp; it < items;
       it += (int64_t)gridDim.x * kBlkWarps) {
    const int r = (int)(it / per_row);
    const int lo = (int)(it % per_row) * kBlkCols, hi = min(a.cols, lo + kBlkCols);
    const int kind = s_new[r], p = a.parents[r];
    int live = 0, fresh = -1;
    if (kind >= kNoBlock && p >= 0) {
      const int blocks = (int)(((int64_t)a.seq_lens[p] + (1 << a.shift) - 1) >> a.shift);
      live = s_first[p] == r ? a.held[p] : blocks;
      if (kind >= 0) fresh = blocks - 1;
    }
    const int32_t* from = a.table + (int64_t)max(p, 0) * a.ld;
    int32_t* to = a.out_table + (int64_t)r * a.ld_out;
#pragma unroll 4
    for (int c = lo + lane; c < hi; c += 32)
      to[c] = c >= live ? -1 : c == fresh ? a.free_blocks[kind] : from[c];
  }
}

// ---- which blocks are in use ---------------------------------------------------
__device__ __forceinline__ int kept_blocks(const ReclaimArgs& a, int r) {
  const int64_t len = max(a.seq_lens[r], 0);
  const int64_t blocks = (len + (1 << a.shift) - 1) >> a.shift;
  return (int)min(blocks, (int64_t)min(max(a.held[r], 0), a.cols));
}
__device__ __forceinline__ void mark(const ReclaimArgs& a, int id) {
  if (id < 0 || id >= a.num_blocks) {
    atomicOr(a.err_word, kErrBadBlock);
    return;
  }
  // (read first: what all rows share would be the same word's atomic again and again)
  uint32_t* word = a.used + (id >> 5);
  const uint32_t bit = 1u << (id & 31);
  if (!(__ldcg(word) & bit)) atomicOr(word, bit);
}

// A warp to 256 columns of a row.
__global__ void __launch_bounds__(kBlkThreads) mark_kernel(ReclaimArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  const int per_row = (a.cols + kBlkCols - 1) / kBlkCols;
  const int64_t items = (int64_t)a.B * per_row;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.n_prefix; i += kBlkThreads) mark(a, a.prefix[i]);
  for (int64_t it = (int64_t)blockIdx.x * kBlkWarps + warp; it < items;
       it += (int64_t)gridDim.x * kBlkWarps) {
    const int r = (int)(it / per_row);
    const int lo = (int)(it % per_row) * kBlkCols, hi = min(a.cols, lo + kBlkCols);
    const int kept = kept_blocks(a, r);
    int32_t* row = a.table + (int64_t)r * a.ld;
    int id[kBlkCols / 32];
#pragma unroll
    for (int i = 0; i < kBlkCols / 32; ++i) {
      const int c = lo + i * 32 + lane;
      id[i] = c < min(hi, kept) ? row[c] : 0;
    }
#pragma unroll
    for (int i = 0; i < kBlkCols / 32; ++i) {
      const int c = lo + i * 32 + lane;
      if (c < min(hi, kept)) mark(a, id[i]);
      else if (c < hi && !a.compact) row[c] = -1;
    }
    if (lo == 0 && lane == 0) a.out_held[r] = kept;
  }
}

// The set bits of words [0, n), and those of words [0, w0), w0 a multiple of 4; of all
// threads together.
__device__ __forceinline__ void count_bits(const uint32_t* used, int64_t n, int64_t w0, int* s,
                                           int* total, int* before) {
  int sum = 0, low = 0;
  const int64_t quads = n / 4;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < quads; i += kBlkThreads) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(used) + i);
    const int bits = __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
    sum += bits;
    low += i * 4 < w0 ? bits : 0;
  }
  for (int64_t i = quads * 4 + threadIdx.x; i < n; i += kBlkThreads) {
    const int bits = __popc(__ldcg(used + i));
    sum += bits;
    low += i < w0 ? bits : 0;
  }
  block_scan_i(sum, s, total);
  block_scan_i(low, s, before);
}

// A CTA to a stretch of words; it counts the words before it, and all of them, itself: for
// 2^20 blocks 128 KB out of L2, which takes less than another launch.  (2048 requests of 512
// columns over 2^20 blocks: 22.8 us in all, which is latency: 6.4 MB.)
//   release: the used ids in order, then the free ones.
//   compact: the i-th used id that is not below n_used = their number moves to the i-th
//   free id below n_used; ranks[w] = the used ids before word w, for the rows' new ids.
__global__ void __launch_bounds__(kBlkThreads) sweep_kernel(ReclaimArgs a) {
  __shared__ int s_scan[kBlkWarps + 1];
  __shared__ uint32_t s_bits[kBlkThreads];
  __shared__ int s_rank[kBlkThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t words = ((int64_t)a.num_blocks + 31) >> 5;
  const int64_t w0 = (int64_t)blockIdx.x * a.share, w1 = min(w0 + a.share, words);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  int n_used, before;
  count_bits(a.used, words, w0, s_scan, &n_used, &before);
  int low = 0;  // used ids below n_used
  if (a.compact) {
    int none;
    count_bits(a.used, n_used >> 5, 0, s_scan, &low, &none);
    if (n_used & 31) low += __popc(__ldcg(a.used + (n_used >> 5)) & ((1u << (n_used & 31)) - 1));
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.out_cursor[0] = n_used;
    if (a.compact) {
      a.count[0] = n_used - low;
      a.totals[0] = n_used;
      a.totals[1] = low;
    }
  }
  for (int64_t base = w0; base < w1; base += kBlkThreads) {
    const int64_t w = base + tid;
    const uint32_t bits = w < w1 ? __ldcg(a.used + w) : 0;
    int total;
    const int rank = before + block_scan_i(__popc(bits), s_scan, &total) - __popc(bits);
    before += total;
    if (a.compact && w < w1) a.ranks[w] = rank;
    __syncthreads();  // (the round before has been read)
    s_bits[tid] = bits;
    s_rank[tid] = rank;
    __syncthreads();
    // a warp to a word, a lane to an id
    const int here = (int)min(w1 - base, (int64_t)kBlkThreads);
#pragma unroll 4
    for (int i = warp; i < here; i += kBlkWarps) {
      const uint32_t m = s_bits[i];
      const int64_t id64 = ((base + i) << 5) + lane;
      const int at = s_rank[i] + __popc(m & ((1u << lane) - 1));
      if (id64 >= a.num_blocks) continue;
      const int id = (int)id64;
      const bool in_use = (m >> lane) & 1;
      if (!a.compact) {
        a.free_blocks[in_use ? at : n_used + id - at] = id;
      } else {
        a.free_blocks[id] = id;
        if (in_use && id >= n_used) a.src[at - low] = id;
        if (!in_use && id < n_used) a.dst[id - at] = id;
        if (id >= n_used - low && id < a.num_blocks / 2) a.src[id] = a.dst[id] = -1;
      }
    }
  }
}

// The rows' and the prefix's new ids.
__device__ __forceinline__ int new_id(const ReclaimArgs& a, int id, int n_used, int low) {
  if (id < 0 || id >= a.num_blocks) return -1;
  if (id < n_used) return id;
  const uint32_t m = __ldcg(a.used + (id >> 5)) & ((1u << (id & 31)) - 1);
  return a.dst[a.ranks[id >> 5] + __popc(m) - low];
}
__global__ void __launch_bounds__(kBlkThreads) renumber_kernel(ReclaimArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per_row = (a.cols + kBlkCols - 1) / kBlkCols;
  const int64_t items = (int64_t)a.B * per_row;
  const int n_used = a.totals[0], low = a.totals[1];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.n_prefix; i += kBlkThreads)
      a.out_prefix[i] = new_id(a, a.prefix[i], n_used, low);
  for (int64_t it = (int64_t)blockIdx.x * kBlkWarps + warp; it < items;
       it += (int64_t)gridDim.x * kBlkWarps) {
    const int r = (int)(it / per_row);
    const int lo = (int)(it % per_row) * kBlkCols, hi = min(a.cols, lo + kBlkCols);
    const int kept = kept_blocks(a, r);
    const int32_t* row = a.table + (int64_t)r * a.ld;
    int32_t* to = a.out_table + (int64_t)r * a.ld_out;
#pragma unroll 4
    for (int c = lo + lane; c < hi; c += 32)
      to[c] = c < kept ? new_id(a, row[c], n_used, low) : -1;
  }
}

// ---- block copies ----------------------------------------------------------------
// Pair i: block src[i] to dst[i] in every cache.  A CTA takes pieces of kPiece units, the
// pieces of a block next to each other.  Bound by the memory: 717 MB read and as many
// written in 213 us (2 layers' K and V; 6.7 TB/s, 0.99 of a plain copy's rate).  What gives
// that is loads under way: 16 of 16 bytes a thread and 32 CTAs an SM, handed out as others
// end, where 8 of each took 224 us.  More CTAs gain nothing and cost those calls whose
// count, known on the device only, is small.
constexpr int kCopyThreads = 256, kAhead = 16, kPiece = kCopyThreads * kAhead;
template <typename U>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
  int n = a.n;
  if (a.count) n = min(n, max(a.count[0], 0));
  const int64_t units = a.block_bytes / (int64_t)sizeof(U);
  const int64_t pieces = (units + kPiece - 1) / kPiece;
  const int64_t each = pieces * a.n_caches;
  for (int64_t it = blockIdx.x; it < each * n; it += gridDim.x) {
    const int i = (int)(it / each);
    const int64_t rest = it - i * each;
    const int c = (int)(rest / pieces);
    const int s = a.src[i], d = a.dst[i];
    if (s < 0 || d < 0) continue;
    if (s >= a.num_blocks || d >= a.num_blocks) {
      if (threadIdx.x == 0) atomicOr(a.err_word, kErrBadBlock);
      continue;
    }
    char* cache = static_cast<char*>(a.caches[c]);
    const U* from = reinterpret_cast<const U*>(cache + s * a.block_stride);
    U* to = reinterpret_cast<U*>(cache + d * a.block_stride);
    const int64_t u0 = (rest - c * pieces) * kPiece + threadIdx.x;
    U v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (u0 + k * kCopyThreads < units) v[k] = from[u0 + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (u0 + k * kCopyThreads < units) to[u0 + k * kCopyThreads] = v[k];
  }
}

int64_t table_items(int rows, int cols) {
  return ((int64_t)rows * ((cols + kBlkCols - 1) / kBlkCols) + kBlkWarps - 1) / kBlkWarps;
}

}  // namespace

cudaError_t prepare_blocks() {
  return cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(int32_t) * 2 * VT_PAGED_MAX_BATCH);
}

cudaError_t launch_fork(const ForkArgs& a, int num_sms, cudaStream_t stream) {
  int64_t grid = table_items(a.R, a.cols);
  if (grid > num_sms) grid = num_sms;
  fork_kernel<<<(unsigned)grid, kBlkThreads, sizeof(int32_t) * ((size_t)a.B + a.R), stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_reclaim(ReclaimArgs a, int num_sms, cudaStream_t stream) {
  const int64_t words = ((int64_t)a.num_blocks + 31) / 32;
  cudaError_t e = cudaMemsetAsync(a.used, 0, (size_t)words * 4, stream);
  if (e != cudaSuccess) return e;
  int64_t grid = table_items(a.B, a.cols);
  if (grid > 4 * num_sms) grid = 4 * num_sms;
  mark_kernel<<<(unsigned)grid, kBlkThreads, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // two CTAs an SM, 32 words to each at least
  const int64_t share = (words + 2 * num_sms - 1) / (2 * num_sms);
  a.share = (int32_t)((share + 31) / 32 * 32);
  // (each begins while the one before it ends, and waits for it)
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)((words + a.share - 1) / a.share));
  cfg.blockDim = dim3(kBlkThreads);
  if ((e = cudaLaunchKernelEx(&cfg, sweep_kernel, a)) != cudaSuccess || !a.compact) return e;
  cfg.gridDim = dim3((unsigned)grid);
  return cudaLaunchKernelEx(&cfg, renumber_kernel, a);
}

cudaError_t launch_copy(const CopyArgs& a, bool wide, int num_sms, cudaStream_t stream) {
  const int64_t unit = wide ? 16 : 1;
  const int64_t pieces = (a.block_bytes / unit + kPiece - 1) / kPiece * a.n_caches * a.n;
  const int64_t most = 32ll * num_sms;
  const unsigned grid = (unsigned)(pieces < most ? pieces : most);
  if (wide) copy_kernel<uint4><<<grid, kCopyThreads, 0, stream>>>(a);
  else copy_kernel<unsigned char><<<grid, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace vt
