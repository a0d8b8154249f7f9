// Pieces of the paged caches' tcgen05 kernels: 128 x 128 bf16 tiles in shared memory (two 64-column
// halves, 128-byte swizzle), their matrix descriptors, and a query row's accumulator in TMEM: the tile
// layout of the rolling-window kernel (rkv_attention.cu).
#pragma once

#include "numeric.cuh"
#include "ptx_sm100.cuh"
#include "rkv_internal.h"

namespace rkv {

constexpr int kSlab = 128 * 64 * 2;  // 128 rows x 64 bf16, one 128-byte swizzle span per row
constexpr int kTile = 2 * kSlab;     // 128 rows x 128 bf16

// K-major operand (Q or K tile): k-step kk covers elements [16kk, 16kk+16) of every row.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t tile_addr, int kk) {
  return ptx::smem_desc_sw128(tile_addr + (kk >> 2) * kSlab + (kk & 3) * 32, 16, 1024);
}

// MN-major operand (V tile as B of O += P V): k-step kk covers keys [16kk, 16kk+16);
// the two 64-column halves of d are kSlab apart.
__device__ __forceinline__ uint64_t desc_v(uint32_t tile_addr, int kk) {
  return ptx::smem_desc_sw128(tile_addr + kk * 2048, kSlab, 1024);
}

// two fp32 -> packed bf16x2 (lo in the low half), round to nearest even, one conversion
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// O (this thread's row, 128 fp32 TMEM columns at tO) *= f
__device__ __forceinline__ void scale_o(uint32_t tO, float f) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t rr[32];
    ptx::tmem_ld32(tO + 32 * c, rr);
#pragma unroll
    for (int i = 0; i < 32; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * f);
    ptx::tmem_st32(tO + 32 * c, rr);
  }
}

}  // namespace rkv
