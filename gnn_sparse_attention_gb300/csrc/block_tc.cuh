// block_tc.cuh -- what the tensor-core block-attention kernels share: barrier
// and TMA helpers, tile numbering, and the operand tensor maps.
#pragma once

#include <cuda.h>

#include "block.cuh"
#include "tcgen05.cuh"

namespace gattn {
namespace tc {

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

// Whether the phase of this parity is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait of a whole warp: the same answer in every lane, so that a wait
// that gives up takes the warp out of its loop together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          uint32_t limit = kWaitLimit) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit));
}

__device__ __forceinline__ void tma_tile3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_alloc512(uint32_t* slot) {  // one whole warp
  asm volatile(
      "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(slot))
      : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_free512(uint32_t addr) {  // one whole warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(addr) : "memory");
}

// D[128][N] (+)= A[128][K] B[N][K]^T, bf16 operands of K = 64 KB columns in
// 128-byte swizzled tiles [K / 64][rows][128 B]; both K-major.
template <int KB>
__device__ __forceinline__ void mma_kk(uint32_t d, const uint8_t* a, int a_piece, const uint8_t* b,
                                       int b_piece, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < 4 * KB; ++k)
    mma_bf16(d, sw128_desc(smem_u32(a + (k / 4) * a_piece) + (k % 4) * 32, 16, 1024),
             sw128_desc(smem_u32(b + (k / 4) * b_piece) + (k % 4) * 32, 16, 1024), idesc, k > 0);
}

// D[128][N] (+)= A[128][K] B[K][N]: A K-major tiles [K / 64][128][128 B], B as
// loaded row by row, [N / 64][K rows][128 B] (MN-major: 64-column pieces
// b_piece bytes apart, groups of 8 rows 1024 bytes apart).
template <int K>
__device__ __forceinline__ void mma_km(uint32_t d, const uint8_t* a, int a_piece, const uint8_t* b,
                                       int b_piece, uint32_t idesc, bool add) {
#pragma unroll
  for (int k = 0; k < K / 16; ++k)
    mma_bf16(d, sw128_desc(smem_u32(a + (k / 4) * a_piece) + (k % 4) * 32, 16, 1024),
             sw128_desc(smem_u32(b) + k * 2048, b_piece, 1024), idesc, (add || k > 0) ? 1u : 0u);
}

// The same with A in TMEM: lane r holds row r, a 32-bit column two consecutive
// bf16 of K.  The K columns sit in groups of `group` bf16, `stride` TMEM columns
// apart (a thread overwrites the scores that it has read).
template <int K>
__device__ __forceinline__ void mma_tm(uint32_t d, uint32_t a, int group, int stride,
                                       const uint8_t* b, int b_piece, uint32_t idesc, bool add) {
#pragma unroll
  for (int k = 0; k < K / 16; ++k) {
    const uint32_t at = a + (k * 16 / group) * stride + (k * 16 % group) / 2;
    const uint64_t bd = sw128_desc(smem_u32(b) + k * 2048, b_piece, 1024);
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(at), "l"(bd), "r"(idesc), "r"((add || k > 0) ? 1u : 0u)
        : "memory");
  }
}

}  // namespace tc

// Tensor map of [rows][heads][D] bf16 read in boxes of 64 columns (zeros past
// D), `box_heads` heads and `box_rows` rows, 128-byte swizzle.
bool encode_heads_map(CUtensorMap* map, const void* base, int64_t rows, int heads, int D,
                      int box_heads, int box_rows);

size_t block_fwd_tc_workspace(const BlockGeom& g);
gattn_status launch_block_fwd_tc(const BlockGeom& g, const void* Q, const void* K, const void* V,
                                 const int32_t* idx, void* out, float* lse, void* ws,
                                 cudaStream_t st);
gattn_status launch_block_bwd_tc(const BlockBwdParams& p, cudaStream_t st);
// Whether a forward (backward) kernel gave up a bounded wait on this device; clears the record.
cudaError_t block_fwd_tc_take_error(int* err);
cudaError_t block_bwd_tc_take_error(int* err);

}  // namespace gattn
