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
// that gives up takes the warp out of its loop together.  A poll returns after 4 us
// (measured; kSuspendNs asks for more).  A warp may have to wait for a whole work
// item, up to 0.1 s, so it gives up after a second.  What a CTA that gave up has in
// flight lands within microseconds; it waits 20 ms for each.
constexpr uint32_t kRoleLimit = 250000, kDrainLimit = 5000;
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          uint32_t limit = kRoleLimit) {
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

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};\n" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(
          taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// One 32-bit column of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};\n" ::"r"(taddr),
               "r"(__float_as_uint(v))
               : "memory");
}
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {  // (valid after tmem_wait_ld)
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n" : "=r"(r) : "r"(taddr));
  return __uint_as_float(r);
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

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n"
               : "=r"(p));
  return p != 0;
}
// The same value in every lane, known to be so by the compiler: the products'
// descriptors then stay in uniform registers, where a product costs a few
// instructions (built per lane they cost more cycles than the product).
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Descriptor of an operand tile: K-major (swizzled 128-byte rows), and as
// loaded row by row and read along the rows (MN-major; 64-column pieces
// `piece` bytes apart).  Offsets within the tile are added to the address
// field with desc_at.
__device__ __forceinline__ uint64_t desc_k(const void* tile) {
  return sw128_desc(smem_u32(tile), 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mn(const void* tile, int piece) {
  return sw128_desc(smem_u32(tile), piece, 1024);
}
__device__ __forceinline__ uint64_t desc_at(uint64_t d, int bytes) { return d + (bytes >> 4); }

// D[128][N] = A[128][K] B[N][K]^T, bf16 operands of K = 64 KB columns in
// 128-byte swizzled tiles [K / 64][rows][128 B]; both K-major.  One lane.
template <int KB>
__device__ __forceinline__ void mma_kk(uint32_t d, uint64_t a, int a_piece, uint64_t b,
                                       int b_piece, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < 4 * KB; ++k)
    mma_bf16(d, desc_at(a, (k / 4) * a_piece + (k % 4) * 32),
             desc_at(b, (k / 4) * b_piece + (k % 4) * 32), idesc, k > 0);
}

// D[128][N] (+)= A[128][K] B[K][N]: A in TMEM (lane r holds row r, a 32-bit
// column two consecutive bf16 of K), B MN-major.  A's K columns sit in groups of
// `group` bf16, `stride` TMEM columns apart (a thread overwrites the scores
// that it has read).  One lane.
template <int K>
__device__ __forceinline__ void mma_tm(uint32_t d, uint32_t a, int group, int stride, uint64_t b,
                                       uint32_t idesc, bool add) {
#pragma unroll
  for (int k = 0; k < K / 16; ++k) {
    const uint32_t at = a + (k * 16 / group) * stride + (k * 16 % group) / 2;
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(at), "l"(desc_at(b, k * 2048)), "r"(idesc), "r"((add || k > 0) ? 1u : 0u)
        : "memory");
  }
}

// 32 fp32 columns as 16 registers of bf16 pairs
__device__ __forceinline__ void pack_row(const float* v, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = bf16x2_bits(v[2 * i], v[2 * i + 1]);
}
// Packed columns [col, col + 32) of a row of D values at `row`: 32-byte stores
// where the address allows them (a lane then fills a whole sector; 16-byte
// stores to rows far apart take twice the time).
__device__ __forceinline__ void store_packed(__nv_bfloat16* row, int col, int D, const uint32_t* w,
                                             bool wide) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int c = col + q * 16;
    if (c + 16 <= D && wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(row + c),
                   "r"(w[8 * q]), "r"(w[8 * q + 1]), "r"(w[8 * q + 2]), "r"(w[8 * q + 3]),
                   "r"(w[8 * q + 4]), "r"(w[8 * q + 5]), "r"(w[8 * q + 6]), "r"(w[8 * q + 7])
                   : "memory");
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (c + 8 * e < D)
          *reinterpret_cast<uint4*>(row + c + 8 * e) =
              make_uint4(w[8 * q + 4 * e], w[8 * q + 4 * e + 1], w[8 * q + 4 * e + 2],
                         w[8 * q + 4 * e + 3]);
    }
  }
}
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int col, int D, const float* v,
                                          bool wide) {
  uint32_t w[16];
  pack_row(v, w);
  store_packed(row, col, D, w, wide);
}
__device__ __forceinline__ bool wide_rows(const void* base, int D) {
  return D >= 16 && (reinterpret_cast<uintptr_t>(base) & 31) == 0;
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
