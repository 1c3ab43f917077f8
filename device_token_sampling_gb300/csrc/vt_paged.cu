// vt_paged.cu -- the paged-batch entry points of include/vt_sampler.h: block
// tables and slot maps from request lengths, and attention over the cache they
// describe.  Host side only: checks of arguments, launch planning, launches.
// Every buffer is allocated in vt_paged_create.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>

#include "vt_device.cuh"
#include "vt_paged.h"
#include "vt_sampler.h"

struct vt_paged {
  vt_paged_config cfg{};
  char err[512] = "";
  int num_sms = 0;
  int shift = 0;
  int64_t part_rows = 0;  // rows of partial results the workspace holds
  float* d_part_o = nullptr;
  float2* d_part_ml = nullptr;
  int32_t* d_err = nullptr;  // the error word, then the attention's work counter
  int32_t* h_err = nullptr;
  int64_t wait_cycles = vt::kWaitCycles;  // limit of the attention's waits
  cudaStream_t last_stream = nullptr;
  bool launched = false;
};

namespace {

int fail(vt_paged* h, int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(h->err, sizeof h->err, fmt, ap);
  va_end(ap);
  return code;
}

// The handle's device, for the duration of a call.
struct Device {
  int prev = -1;
  bool ok = true;
  explicit Device(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
  }
  ~Device() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

#define VT_TRY(h, expr)                                                                  \
  do {                                                                                   \
    const cudaError_t e_ = (expr);                                                       \
    if (e_ != cudaSuccess)                                                               \
      return fail((h), VT_ERR_CUDA, "%s failed: %s", #expr, cudaGetErrorString(e_));     \
  } while (0)

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool config_ok(const vt_paged_config& c) {
  if (c.max_batch < 1 || c.max_batch > VT_PAGED_MAX_BATCH) return false;
  if (c.block_size < 1 || c.block_size > 1024 || (c.block_size & (c.block_size - 1))) return false;
  if (c.max_blocks < 1 || (int64_t)c.max_blocks * c.block_size > (1ll << 30)) return false;
  if (c.device < 0) return false;
  if (c.q_heads == 0) return c.kv_heads == 0 && c.head_dim == 0;
  if (c.kv_heads < 1 || c.q_heads < c.kv_heads || c.q_heads > 1024 || c.q_heads % c.kv_heads)
    return false;
  return c.head_dim == 64 || c.head_dim == 128;
}

// How a call's work is split.  Units of about 256 tokens keep the warps busy to
// the end and write 2 % of what they read as partial results (128 and 512 tokens
// are 4 % slower on 256 requests of 512 tokens); shorter ones, down to 64 tokens,
// until there are two for every warp (64 requests of 256 tokens: 25 us in units of
// 128 tokens, 29 in units of 170).  The partial results
// have to fit the workspace.
void plan_attention(const vt_paged* h, int B, int prefix_len, int max_len, vt::AttnArgs& a) {
  const int64_t warps = 8ll * h->num_sms;  // of unit_kernel, on the GPU at once
  const int64_t rows = (int64_t)B * a.hq;
  // more than one 16-row tile of rows behind the prefix: the tensor-memory kernel,
  // 256 rows to a CTA, one CTA to an SM (below, that kernel would pad 128-row tiles)
  a.prefix_mma = prefix_len > 0 && (int64_t)B * a.G > 16 && vt::prefix_mma_takes(a);
  // rows of the other units: 8, the width of their MMAs, unless more heads share a
  // kv head or more rows the prefix
  a.unit_rows = a.G > 8 || (prefix_len > 0 && !a.prefix_mma && (int64_t)B * a.G > 8) ? 16 : 8;
  a.prefix_tiles = (int)ceil_div((int64_t)B * a.G, a.prefix_mma ? 128 : a.unit_rows);
  a.own_tiles = (int)ceil_div(a.G, a.unit_rows);
  const int64_t own_len = std::max(1, max_len - (prefix_len & ~15));
  // splits of `len` tokens for `each` units a split
  auto splits = [&](int64_t len, int64_t each) {
    const int64_t fill = ceil_div(2 * warps, each);
    return std::clamp<int64_t>(std::max(fill, ceil_div(len, 256)), 1, ceil_div(len, 64));
  };
  const int step = a.prefix_mma ? 128 : 64;  // tokens a prefix split is a multiple of
  int64_t sp = 0;
  if (a.prefix_mma)  // so that the grid is one round of CTAs
    sp = std::clamp<int64_t>(h->num_sms / std::max<int64_t>(1, ceil_div(a.prefix_tiles, 2) * a.hkv),
                             1, std::min<int64_t>(64, ceil_div(prefix_len, step)));
  else if (prefix_len > 0)
    sp = std::min<int64_t>(64, splits(prefix_len, (int64_t)a.prefix_tiles * a.hkv));
  int64_t so = std::min<int64_t>(64, splits(own_len, (int64_t)a.own_tiles * a.hkv * B));
  while ((sp + so) * rows > h->part_rows && (sp > 1 || so > 1)) {
    if (sp >= so) --sp;
    else --so;
  }
  a.prefix_splits = a.prefix_chunk = 0;
  if (sp > 0) {
    a.prefix_chunk = (int)ceil_div(ceil_div(prefix_len, sp), step) * step;
    a.prefix_splits = (int)ceil_div(prefix_len, a.prefix_chunk);
  }
  a.own_splits = (int)so;
  a.own_chunk = (int)ceil_div(ceil_div(own_len, so), 16) * 16;
}

void free_paged(vt_paged* h) {
  if (h->d_part_o) cudaFree(h->d_part_o);
  if (h->d_part_ml) cudaFree(h->d_part_ml);
  if (h->d_err) cudaFree(h->d_err);
  if (h->h_err) cudaFreeHost(h->h_err);
  delete h;
}

}  // namespace

int vt_paged_create(const vt_paged_config* config, vt_paged** out) {
  if (!config || !out || !config_ok(*config)) return VT_ERR_INVALID_ARG;
  vt_paged* h = new (std::nothrow) vt_paged;
  if (!h) return VT_ERR_CUDA;
  h->cfg = *config;
  while ((1 << h->shift) < config->block_size) ++h->shift;
  // (for the test of this failure path: the waits count as run out)
  const char* fault = std::getenv("VT_FAULT_INJECT");
  if (fault && std::strcmp(fault, "wait") == 0) h->wait_cycles = 0;
  Device guard(config->device);
  cudaDeviceProp prop;
  bool ok = guard.ok && cudaGetDeviceProperties(&prop, config->device) == cudaSuccess &&
            prop.major == 10 && prop.minor == 3;  // built for sm_103a only
  if (ok) {
    h->num_sms = prop.multiProcessorCount;
    ok = vt::prepare_tables() == cudaSuccess && vt::prepare_prefix_attention() == cudaSuccess &&
         cudaMalloc(&h->d_err, 2 * sizeof(int32_t)) == cudaSuccess &&
         cudaMemset(h->d_err, 0, 2 * sizeof(int32_t)) == cudaSuccess &&
         cudaMallocHost(&h->h_err, sizeof(int32_t)) == cudaSuccess;
  }
  if (ok && config->q_heads > 0) {
    h->part_rows = 8ll * config->max_batch * config->q_heads + 32768;
    ok = cudaMalloc(&h->d_part_o, h->part_rows * config->head_dim * sizeof(float)) ==
             cudaSuccess &&
         cudaMalloc(&h->d_part_ml, h->part_rows * sizeof(float2)) == cudaSuccess;
  }
  if (!ok) {
    free_paged(h);
    cudaGetLastError();
    return VT_ERR_CUDA;
  }
  *out = h;
  return VT_OK;
}

void vt_paged_destroy(vt_paged* h) {
  if (!h) return;
  Device guard(h->cfg.device);
  if (h->launched) cudaStreamSynchronize(h->last_stream);
  free_paged(h);
}

const char* vt_paged_last_error(const vt_paged* h) { return h ? h->err : "null handle"; }

int vt_paged_check_errors(vt_paged* h) {
  if (!h) return VT_ERR_INVALID_ARG;
  Device guard(h->cfg.device);
  if (!guard.ok) return fail(h, VT_ERR_CUDA, "cannot select device %d", h->cfg.device);
  VT_TRY(h, cudaStreamSynchronize(h->last_stream));
  VT_TRY(h, cudaMemcpy(h->h_err, h->d_err, sizeof(int32_t), cudaMemcpyDeviceToHost));
  if (*h->h_err == 0) return VT_OK;
  VT_TRY(h, cudaMemset(h->d_err, 0, sizeof(int32_t)));
  if (*h->h_err & vt::kErrTimeout)
    return fail(h, VT_ERR_TIMEOUT, "a bounded device wait ran out");
  return fail(h, VT_ERR_INVALID_ARG, "a block id outside the cache was met; its tokens were "
                                     "left out");
}

int vt_paged_tables(vt_paged* h, int32_t B, const int32_t* seq_lens, const int32_t* query_lens,
                    const int32_t* held, const int32_t* prefix_blocks, int32_t num_prefix_blocks,
                    const int32_t* free_blocks, int32_t num_free, const int32_t* cursor,
                    int32_t* table, int64_t ld_table, int32_t* out_held, int32_t* out_cursor,
                    int32_t* out_starts, int64_t* out_slots, int32_t* out_positions,
                    int64_t capacity, int32_t* out_status, void* stream) {
  if (!h) return VT_ERR_INVALID_ARG;
  if (B < 1) return fail(h, VT_ERR_INVALID_ARG, "B=%d: need B >= 1", B);
  if (B > h->cfg.max_batch)
    return fail(h, VT_ERR_CAPACITY, "B=%d above max_batch=%d", B, h->cfg.max_batch);
  if (!seq_lens || !query_lens || !cursor || !table || !out_held || !out_cursor || !out_starts ||
      !out_status)
    return fail(h, VT_ERR_INVALID_ARG, "a null array");
  if (num_prefix_blocks < 0 || (num_prefix_blocks > 0 && !prefix_blocks))
    return fail(h, VT_ERR_INVALID_ARG, "num_prefix_blocks=%d with %s prefix blocks",
                num_prefix_blocks, prefix_blocks ? "its" : "no");
  if (num_free < 0 || (num_free > 0 && !free_blocks))
    return fail(h, VT_ERR_INVALID_ARG, "num_free=%d with %s free list", num_free,
                free_blocks ? "its" : "no");
  if (capacity < 0 || capacity > 0x7fffffffll ||
      (capacity > 0 && (!out_slots || !out_positions)))
    return fail(h, VT_ERR_INVALID_ARG, "capacity=%lld outside [0, 2^31) or null slot map",
                (long long)capacity);
  if (ld_table < h->cfg.max_blocks)
    return fail(h, VT_ERR_INVALID_ARG, "ld_table=%lld below max_blocks=%d", (long long)ld_table,
                h->cfg.max_blocks);
  if (out_held == held || out_cursor == cursor)
    return fail(h, VT_ERR_INVALID_ARG, "held and cursor are not updated in place");
  Device guard(h->cfg.device);
  if (!guard.ok) return fail(h, VT_ERR_CUDA, "cannot select device %d", h->cfg.device);
  vt::TablesArgs a;
  std::memset(&a, 0, sizeof a);
  a.B = B;
  a.shift = h->shift;
  a.cols = h->cfg.max_blocks;
  a.ld = ld_table;
  a.table = table;
  a.seq_lens = seq_lens;
  a.query_lens = query_lens;
  a.held = held;
  a.prefix = prefix_blocks;
  a.n_prefix = num_prefix_blocks;
  a.free_blocks = free_blocks;
  a.n_free = num_free;
  a.cursor = cursor;
  a.out_held = out_held;
  a.out_cursor = out_cursor;
  a.starts = out_starts;
  a.slots = out_slots;
  a.positions = out_positions;
  a.capacity = capacity;
  a.status = out_status;
  a.vec = aligned(out_slots, 16) && aligned(out_positions, 16);
  cudaStream_t st = (cudaStream_t)stream;
  VT_TRY(h, vt::launch_tables(a, h->num_sms, st));
  h->last_stream = st;
  h->launched = true;
  h->err[0] = 0;
  return VT_OK;
}

int vt_paged_attention_ex(vt_paged* h, int32_t dtype, int32_t B, const void* q, int64_t q_row,
                          int64_t q_head, const void* k_cache, const void* v_cache,
                          int32_t num_blocks, int64_t block_stride, int64_t token_stride,
                          int64_t head_stride, const int32_t* table, int64_t ld_table,
                          int32_t table_cols, const int32_t* seq_lens,
                          const int32_t* prefix_blocks, int32_t prefix_len, int32_t max_seq_len,
                          float scale, void* out, float* out_lse, void* stream) {
  if (!h) return VT_ERR_INVALID_ARG;
  const vt_paged_config& c = h->cfg;
  if (c.q_heads == 0)
    return fail(h, VT_ERR_STATE, "the handle was created for tables alone (q_heads=0)");
  if (dtype != VT_DTYPE_BF16 && dtype != VT_DTYPE_F16)
    return fail(h, VT_ERR_INVALID_ARG, "dtype %d: need bf16 or fp16", dtype);
  if (B < 1) return fail(h, VT_ERR_INVALID_ARG, "B=%d: need B >= 1", B);
  if (B > c.max_batch) return fail(h, VT_ERR_CAPACITY, "B=%d above max_batch=%d", B, c.max_batch);
  if (!q || !k_cache || !v_cache || !table || !seq_lens || !out)
    return fail(h, VT_ERR_INVALID_ARG, "a null array");
  const int64_t cap = (int64_t)c.max_blocks * c.block_size;
  if (prefix_len < 0 || prefix_len > cap)
    return fail(h, VT_ERR_INVALID_ARG, "prefix_len=%d outside [0, %lld]", prefix_len,
                (long long)cap);
  if (prefix_len > 0 && !prefix_blocks)
    return fail(h, VT_ERR_INVALID_ARG, "prefix_len=%d without prefix blocks", prefix_len);
  if (num_blocks < 1 || ld_table < 1 || table_cols < 1)
    return fail(h, VT_ERR_INVALID_ARG, "num_blocks=%d, ld_table=%lld, table_cols=%d: need at least 1",
                num_blocks, (long long)ld_table, table_cols);
  if (max_seq_len < 0) return fail(h, VT_ERR_INVALID_ARG, "max_seq_len=%d", max_seq_len);
  if (!std::isfinite(scale)) return fail(h, VT_ERR_INVALID_ARG, "scale is not finite");
  // rows are copied 16 bytes at a time
  if ((q_row | q_head | block_stride | token_stride | head_stride) % 8 ||
      !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return fail(h, VT_ERR_INVALID_ARG,
                "arrays must start on 16 bytes and strides be multiples of 8 elements");
  Device guard(c.device);
  if (!guard.ok) return fail(h, VT_ERR_CUDA, "cannot select device %d", c.device);
  vt::AttnArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = q;
  a.q_row = q_row;
  a.q_head = q_head;
  a.k = k_cache;
  a.v = v_cache;
  a.block_stride = block_stride;
  a.token_stride = token_stride;
  a.head_stride = head_stride;
  a.num_blocks = num_blocks;
  a.shift = h->shift;
  a.table = table;
  a.ld_table = ld_table;
  a.seq_lens = seq_lens;
  a.prefix_blocks = prefix_blocks;
  a.prefix_len = prefix_len;
  a.cols = std::min(c.max_blocks, table_cols);
  a.B = B;
  a.hq = c.q_heads;
  a.hkv = c.kv_heads;
  a.G = c.q_heads / c.kv_heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  const int64_t longest = (int64_t)a.cols * c.block_size;
  plan_attention(h, B, prefix_len,
                 (int)(max_seq_len > 0 ? std::min<int64_t>(max_seq_len, longest) : longest), a);
  a.part_o = h->d_part_o;
  a.part_ml = h->d_part_ml;
  a.out = out;
  a.lse = out_lse;
  a.work = h->d_err + 1;
  a.num_sms = h->num_sms;
  a.err_word = h->d_err;
  a.wait_cycles = h->wait_cycles;
  cudaStream_t st = (cudaStream_t)stream;
  VT_TRY(h, vt::launch_prefix_attention(a, dtype, c.head_dim, st));
  h->last_stream = st;
  h->launched = true;
  h->err[0] = 0;
  return VT_OK;
}

int vt_paged_attention(vt_paged* h, int32_t dtype, int32_t B, const void* q, int64_t q_row,
                       int64_t q_head, const void* k_cache, const void* v_cache,
                       int32_t num_blocks, int64_t block_stride, int64_t token_stride,
                       int64_t head_stride, const int32_t* table, int64_t ld_table,
                       const int32_t* seq_lens, const int32_t* prefix_blocks, int32_t prefix_len,
                       int32_t max_seq_len, float scale, void* out, float* out_lse,
                       void* stream) {
  return vt_paged_attention_ex(h, dtype, B, q, q_row, q_head, k_cache, v_cache, num_blocks,
                               block_stride, token_stride, head_stride, table, ld_table,
                               (int32_t)std::min<int64_t>(ld_table, 0x7fffffff), seq_lens,
                               prefix_blocks, prefix_len, max_seq_len, scale, out, out_lse, stream);
}
