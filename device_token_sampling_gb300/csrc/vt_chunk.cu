// vt_chunk.cu -- attention of a chunk of new tokens a request over its paged cache.
//
// Request b has n_b query tokens, the last n_b of its len_b tokens.  Row i of them, of
// head h, is out = sum_j p_j v_j / sum_j p_j over the positions j <= len_b - n_b + i, with
// p_j = exp(scale q . k_j - max).
//
// This file: rows one at a time, in fp32, for layouts that no tensor map holds: q or
// caches with a stride of 0 (broadcast heads, say) or less.  A warp a row reads all of its
// keys and values itself: 1024 tokens of 32 heads take 1.8 ms, on the tensor cores 25 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vt_device.cuh"
#include "vt_paged.h"
#include "vt_sampler.h"

namespace vt {
namespace {

constexpr int kRowWarps = 8;

template <typename T>
__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]);
template <>
__device__ __forceinline__ void widen8<__nv_bfloat16>(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void widen8<__half>(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Whether request b's rows of q are there.
__device__ __forceinline__ bool rows_fine(const ChunkArgs& a, int b) {
  const int s0 = a.starts[b], s1 = a.starts[b + 1];
  return s0 >= 0 && s0 <= s1 && s1 <= a.T;
}

// The request that holds token t: the last b with starts[b] <= t, if t is below its end.
__device__ __forceinline__ int request_of(const int32_t* starts, int B, int64_t t) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid;
  }
  return starts[lo] <= t && t < starts[lo + 1] ? lo : -1;
}

// A warp to a row: a lane to a token for the scores, then a lane to D / 32 elements for
// the product with V.
template <typename T, int D>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(ChunkArgs a) {
  constexpr int W = D / 32;
  __shared__ float s_q[kRowWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rows = (int64_t)a.T * a.hq;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += kRowWarps * 32)
      if (!rows_fine(a, b)) atomicOr(a.err_word, kErrBadRows);
  for (int64_t row = (int64_t)blockIdx.x * kRowWarps + warp; row < rows;
       row += (int64_t)gridDim.x * kRowWarps) {
    const int64_t t = row / a.hq;
    const int head = (int)(row % a.hq);
    const int b = request_of(a.starts, a.B, t);
    if (b < 0 || !rows_fine(a, b)) continue;
    const int s0 = a.starts[b], n = a.starts[b + 1] - s0;
    const int64_t seen = (int64_t)a.seq_lens[b] - n + (t - s0) + 1;
    const int lim = (int)min(max(seen, (int64_t)0), (int64_t)a.cols << a.shift);
    const T* q = static_cast<const T*>(a.q) + t * a.q_row + head * a.q_head;
    __syncwarp();
    for (int i = lane; i < D; i += 32) s_q[warp][i] = static_cast<float>(q[i]) * a.scale_log2;
    __syncwarp();
    const int32_t* table = a.table + (int64_t)b * a.ld_table;
    const int64_t col = head / a.G * a.head_stride;
    float m = -INFINITY, l = 0.f, acc[W] = {};
#pragma unroll 1
    for (int j0 = 0; j0 < lim; j0 += 32) {
      const int j = j0 + lane;
      const int blk = j < lim ? table[j >> a.shift] : -1;
      const bool fine = blk >= 0 && blk < a.num_blocks;
      if (j < lim && !fine) atomicOr(a.err_word, kErrBadBlock);
      const int64_t at =
          fine ? blk * a.block_stride + (j & ((1 << a.shift) - 1)) * a.token_stride + col : 0;
      float s = -INFINITY;
      if (fine) {
        const uint4* k = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + at);
        s = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          float x[8];
          widen8<T>(k[c], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) s += x[i] * s_q[warp][c * 8 + i];
        }
      }
      const float mn = fmaxf(m, warp_max(s)), base = mn == -INFINITY ? 0.f : mn;
      const float f = ex2_approx(m - base), p = ex2_approx(s - base);
      m = mn;
      l = l * f + p;
#pragma unroll
      for (int w = 0; w < W; ++w) acc[w] *= f;
      for (unsigned left = __ballot_sync(0xffffffffu, fine); left; left &= left - 1) {
        const int i = __ffs(left) - 1;
        const float pi = __shfl_sync(0xffffffffu, p, i);
        const T* v = static_cast<const T*>(a.v) + __shfl_sync(0xffffffffu, at, i) + lane * W;
#pragma unroll
        for (int w = 0; w < W; ++w) acc[w] += pi * static_cast<float>(v[w]);
      }
    }
    l = warp_sum_f(l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* out = static_cast<T*>(a.out) + row * D + lane * W;
#pragma unroll
    for (int w = 0; w < W; ++w) out[w] = static_cast<T>(acc[w] * inv);
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
  }
}

template <typename T, int D>
cudaError_t launch_rows(const ChunkArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.T * a.hq, ctas = (rows + kRowWarps - 1) / kRowWarps;
  const int64_t most = 64ll * a.num_sms;
  rows_kernel<T, D><<<(unsigned)(ctas < most ? ctas : most), kRowWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk(const ChunkArgs& a, int dtype, int head_dim, cudaStream_t stream) {
  if (chunk_mma_takes(a)) return launch_chunk_mma(a, dtype, head_dim, stream);
  if (dtype == VT_DTYPE_BF16)
    return head_dim == 128 ? launch_rows<__nv_bfloat16, 128>(a, stream)
                           : launch_rows<__nv_bfloat16, 64>(a, stream);
  return head_dim == 128 ? launch_rows<__half, 128>(a, stream)
                         : launch_rows<__half, 64>(a, stream);
}

}  // namespace vt
