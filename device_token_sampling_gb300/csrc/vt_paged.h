// vt_paged.h -- internal interface between the paged-batch host code and its
// kernels (block tables and slot maps; attention behind a shared prefix).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vt {

constexpr int kErrBadBlock = 4;  // error word: a block id outside the cache was met
constexpr int kErrBadRows = 8;   // a request's starts are not 0 <= first <= end <= T

// ---- block tables and slot maps (vt_tables.cu) -------------------------------
struct TablesArgs {
  int32_t B;
  int32_t shift;               // log2 of the block size
  int32_t cols;                // columns a table row may use
  int64_t ld;                  // table row stride
  int32_t* table;
  const int32_t* seq_lens;     // [B]
  const int32_t* query_lens;   // [B]
  const int32_t* held;         // [B], or null: a new table
  const int32_t* prefix;       // [n_prefix]
  int32_t n_prefix;
  const int32_t* free_blocks;  // [n_free]
  int32_t n_free;
  const int32_t* cursor;       // [1]
  int32_t* out_held;           // [B]
  int32_t* out_cursor;         // [1]
  int32_t* starts;             // [B + 1]
  int64_t* slots;              // [capacity]
  int32_t* positions;          // [capacity]
  int64_t capacity;
  int32_t* status;             // [B]
  int32_t vec;                 // slots and positions 16-byte aligned
  int32_t share;               // filled by launch_tables
};
cudaError_t launch_tables(TablesArgs a, int num_sms, cudaStream_t stream);

// ---- forks, released and compacted blocks, block copies (vt_blocks.cu) --------
struct ForkArgs {
  int32_t R, B;                // rows of the new and of the old table
  int32_t shift, cols;
  const int32_t* parents;      // [R]
  const int32_t* table;        // [B][ld]
  int64_t ld;
  const int32_t* held;         // [B]
  const int32_t* seq_lens;     // [B]
  const int32_t* free_blocks;  // [n_free]
  int32_t n_free;
  const int32_t* cursor;       // [1]
  int32_t* out_table;          // [R][ld_out]
  int64_t ld_out;
  int32_t* out_held;           // [R]
  int32_t* out_seq;            // [R]
  int32_t* out_cursor;         // [1]
  int32_t* src;                // [R]
  int32_t* dst;                // [R]
  int32_t* status;             // [R]
};
cudaError_t launch_fork(const ForkArgs& a, int num_sms, cudaStream_t stream);

struct ReclaimArgs {
  int32_t B, shift, cols, num_blocks;
  int32_t compact;             // else release
  int32_t* table;              // [B][ld]
  int64_t ld;
  const int32_t* held;         // [B]
  const int32_t* seq_lens;     // [B]
  const int32_t* prefix;       // [n_prefix]
  int32_t n_prefix;
  int32_t* out_held;           // [B]
  int32_t* free_blocks;        // [num_blocks]
  int32_t* out_cursor;         // [1]
  // compact alone
  int32_t* out_table;          // [B][ld_out]; may be the table
  int64_t ld_out;
  int32_t* out_prefix;         // [n_prefix]
  int32_t* src;                // [num_blocks / 2]
  int32_t* dst;
  int32_t* count;              // [1]
  // scratch: a bit to a block; the used ids before each word; their number and how
  // many of them are below it
  uint32_t* used;
  int32_t* ranks;
  int32_t* totals;
  int32_t* err_word;
  int32_t share;               // words to a CTA; filled by launch_reclaim
};
cudaError_t launch_reclaim(ReclaimArgs a, int num_sms, cudaStream_t stream);

constexpr int kCopyCaches = 64;  // caches of a launch
struct CopyArgs {
  void* caches[kCopyCaches];
  int32_t n_caches, num_blocks;
  int64_t block_stride, block_bytes;
  const int32_t* src;          // [n]
  const int32_t* dst;
  int32_t n;
  const int32_t* count;        // [1] or null
  int32_t* err_word;
};
// wide: pointers, stride and size are multiples of 16 bytes
cudaError_t launch_copy(const CopyArgs& a, bool wide, int num_sms, cudaStream_t stream);
cudaError_t prepare_blocks();

// ---- attention behind a shared prefix (vt_prefix.cu) -------------------------
struct AttnArgs {
  const void* q;               // [B] rows of q_row elements, heads q_head apart
  int64_t q_row, q_head;
  const void* k;               // cache: block, token and head strides in elements
  const void* v;
  int64_t block_stride, token_stride, head_stride;
  int32_t num_blocks;
  int32_t shift;               // log2 of the block size
  const int32_t* table;        // [B][ld_table]
  int64_t ld_table;
  const int32_t* seq_lens;     // [B]
  const int32_t* prefix_blocks;
  int32_t prefix_len;
  int32_t cols;                // table columns a row may use
  int32_t B, hq, hkv, G;       // G = hq / hkv
  float scale_log2;            // scale * log2(e)
  // the work: prefix units first, then the requests' own units
  int32_t prefix_mma;          // the prefix runs on prefix_kernel, 128 rows to a tile
  int32_t unit_rows;           // rows of unit_kernel's units: 8 or 16
  int32_t prefix_tiles;        // row tiles (unit_rows or 128 rows) of one kv head's B * G rows
  int32_t prefix_splits, prefix_chunk;  // splits of [0, prefix_len), tokens in each
  int32_t own_tiles;           // unit_rows-row tiles of G heads
  int32_t own_splits, own_chunk;
  float* part_o;               // [splits][B * hq][d] fp32, not normalised
  float2* part_ml;             // [splits][B * hq] (max in log2 units, sum)
  void* out;                   // [B][hq][d]
  float* lse;                  // [B][hq] or null
  int32_t* work;               // units taken; 0 between calls
  int32_t num_sms;
  int32_t* err_word;
  int64_t wait_cycles;         // limit of prefix_kernel's waits; 0: they have run out
};
// dtype as VT_DTYPE_BF16 / VT_DTYPE_F16; head_dim 64 or 128.
cudaError_t launch_prefix_attention(const AttnArgs& a, int dtype, int head_dim,
                                    cudaStream_t stream);
// ---- attention of chunks (vt_chunk.cu) -------------------------------------------
struct ChunkStart {  // where a CTA's share of the steps begins
  int64_t at;                  // what the steps in front of it cost
  int32_t b, unit, head, step; // its first unit, and the step in that
  int32_t rounds;              // whole units that the CTA has before
};
struct ChunkArgs {
  const void* q;               // [T] rows of q_row elements, heads q_head apart
  int64_t q_row, q_head;
  const void* k;               // cache: block, token and head strides in elements
  const void* v;
  int64_t block_stride, token_stride, head_stride;
  int32_t num_blocks;
  int32_t shift;               // log2 of the block size
  const int32_t* table;        // [B][ld_table]
  int64_t ld_table;
  int32_t cols;                // table columns a row may use
  const int32_t* starts;       // [B + 1]
  const int32_t* seq_lens;     // [B]
  int32_t B, T, hq, hkv, G;    // G = hq / hkv
  float scale_log2;            // scale * log2(e)
  void* out;                   // [T][hq][d]
  float* lse;                  // [T][hq] or null
  int32_t num_sms;
  int32_t* err_word;
  int64_t wait_cycles;         // limit of the waits; 0: they have run out
  // the tensor cores' way
  int32_t grid;                // CTAs
  int64_t* plan_first;         // [B + 1][2] units and costs in front of each request
  ChunkStart* plan_start;      // [grid + 1]
  int32_t* plan_count;         // [grid][2][4] parts of a unit's rows that are there
  float* part_o;               // [grid][2][256][d] fp32, not normalised
  float2* part_ml;             // [grid][2][256] (max in log2 units, sum)
  // filled by launch_chunk_mma: heads of a tile, parts of the G, tokens of a tile, virtual
  // heads (hkv * parts), bytes of a tile of q
  int32_t heads, parts, tokens, heads_all;
  uint32_t q_bytes;
  int32_t out_wide;            // out starts on 32 bytes
};
cudaError_t launch_chunk(const ChunkArgs& a, int dtype, int head_dim, cudaStream_t stream);
// On the tensor cores (vt_chunk_mma.cu): whether the caches' layout can be taken, the
// launch, and the rows of partial results that `grid` CTAs leave.
bool chunk_mma_takes(const ChunkArgs& a);
cudaError_t launch_chunk_mma(ChunkArgs a, int dtype, int head_dim, cudaStream_t stream);
int64_t chunk_part_rows(int grid);
cudaError_t prepare_chunk();

// Kernel attributes, once for the current device.
cudaError_t prepare_tables();
cudaError_t prepare_prefix_attention();
cudaError_t prepare_prefix_mma();
// The prefix's part of it (vt_prefix_mma.cu): whether its layout can be taken, and
// the launch.
bool prefix_mma_takes(const AttnArgs& a);
cudaError_t launch_prefix_mma(const AttnArgs& a, int dtype, int head_dim, cudaStream_t stream);

}  // namespace vt
