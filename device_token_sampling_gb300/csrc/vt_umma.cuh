// vt_umma.cuh -- what the kernels on the 5th-generation tensor cores share: inline
// PTX of tcgen05 and of tensor copies, bounded waits, and tensor maps of a paged cache.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "vt_device.cuh"
#include "vt_sampler.h"

namespace vt {
namespace {

constexpr int kTileRows = 128;
constexpr int kTileTokens = 128;  // of a K or V tile

// Shared memory descriptors: start address, leading and stride byte offsets in
// 16-byte units; descriptor version 1; 128-byte swizzle.  Only the low word moves
// from one MMA to the next.
__device__ __forceinline__ constexpr uint32_t desc_hi(uint32_t sbo) {
  return (sbo >> 4) | (1u << 14) | (2u << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3ffff) >> 4) | ((lbo >> 4) << 16);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                       uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
// One lane of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

#define VT_R8(r, i)                                                                       \
  "=r"((r)[i]), "=r"((r)[i + 1]), "=r"((r)[i + 2]), "=r"((r)[i + 3]), "=r"((r)[i + 4]),   \
      "=r"((r)[i + 5]), "=r"((r)[i + 6]), "=r"((r)[i + 7])
#define VT_I8(r, i)                                                                   \
  "r"((r)[i]), "r"((r)[i + 1]), "r"((r)[i + 2]), "r"((r)[i + 3]), "r"((r)[i + 4]),    \
      "r"((r)[i + 5]), "r"((r)[i + 6]), "r"((r)[i + 7])
// 32 columns of this thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : VT_R8(r, 0), VT_R8(r, 8), VT_R8(r, 16), VT_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      VT_I8(r, 0), VT_I8(r, 8), VT_I8(r, 16), VT_I8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Registers that a load has filled are not used before this point.
#define VT_P8(r, i)                                                                       \
  "+r"((r)[i]), "+r"((r)[i + 1]), "+r"((r)[i + 2]), "+r"((r)[i + 3]), "+r"((r)[i + 4]),   \
      "+r"((r)[i + 5]), "+r"((r)[i + 6]), "+r"((r)[i + 7])
__device__ __forceinline__ void loaded(uint32_t (&r)[32]) {
  asm volatile("" : VT_P8(r, 0), VT_P8(r, 8), VT_P8(r, 16), VT_P8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                         int d, int token, int head, int block) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_addr(bar)), "r"(d), "r"(token), "r"(head), "r"(block)
      : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A wait of at most `limit` cycles; with 0 it has run out.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t phase, long long limit) {
  return limit > 0 && mbar_wait_clocked(bar, phase, limit);
}
// The whole warp's: it runs out for all lanes or for none, so that they leave their
// loops together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase, long long limit) {
  return __all_sync(0xffffffffu, wait_for(bar, phase, limit));
}
constexpr long long kDrainCycles = 200000000ll;  // for what is in flight after a run-out

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

[[maybe_unused]] EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A cache as [block][head][token][element], copied kTileTokens tokens (or a block) of 64
// elements at a time.
[[maybe_unused]] bool cache_map(CUtensorMap* map, const void* cache, int dtype, int head_dim,
                                int shift, int kv_heads, int num_blocks, int64_t block_stride,
                                int64_t token_stride, int64_t head_stride) {
  const cuuint64_t dims[4] = {(cuuint64_t)head_dim, 1ull << shift, (cuuint64_t)kv_heads,
                              (cuuint64_t)num_blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)token_stride * 2, (cuuint64_t)head_stride * 2,
                                 (cuuint64_t)block_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)(shift < 7 ? 1 << shift : kTileTokens), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return encode_tiled()(map,
                        dtype == VT_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        4, const_cast<void*>(cache), dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Whether a tensor map can hold the cache: strides in range.
[[maybe_unused]] bool cache_map_takes(int64_t block_stride, int64_t token_stride,
                                      int64_t head_stride) {
  const int64_t most = 1ll << 38;
  return block_stride > 0 && token_stride > 0 && head_stride > 0 &&
         block_stride < most && token_stride < most && head_stride < most &&
         encode_tiled() != nullptr;
}

}  // namespace
}  // namespace vt
