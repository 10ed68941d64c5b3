// Tensor-core pieces shared by the kernels that multiply 4-bit codes: the
// 16 x 8 x 16 half-precision product with fp32 sums, and the split of an fp32
// number into two halves.
//
// The products have 8 to 32 rows on the activation side and each code is used
// once per row, so these kernels live on the rate at which codes arrive from
// memory and become halves in registers; a fifth-generation product would need
// its 128-row operand rebuilt as halves in shared or tensor memory first (four
// times the bytes that arrive), so the warp-level product, which takes the
// decoded registers as they are, is used here.
#pragma once

#include "common.cuh"

namespace sffn {

// d (rows g, g + 8; columns 2t, 2t + 1) += a (16 x 16) b (16 x 8), lane = 4 g + t.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of halves: lane 4 g + t gives row g, columns 2t, 2t + 1.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t h2_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 u32_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }

// hi + lo = (x, y) to 22 bits: hi the nearest half, lo the nearest half of the rest.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = h2_u32(h);
  lo = h2_u32(__floats2half2_rn(x - f.x, y - f.y));
}

// A power of two that brings m > 0 into [2^13, 2^14), and its inverse (m = 0,
// non-finite or below 2^-107: some power of two).
__device__ __forceinline__ void scale_to_half_range(float m, float& up, float& down) {
  const int e = min(max((int)(__float_as_uint(m) >> 23) & 0xff, 20), 254);
  up = __uint_as_float((uint32_t)(267 - e) << 23);
  down = __uint_as_float((uint32_t)(e - 13) << 23);
}

// (w & mask) | 0x6400 in both halves, the exponent of 1024 over the selected
// bits, as the one three-input logic operation that it is.
__device__ __forceinline__ __half2 code_bits(uint32_t w, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
  return u32_h2(r);
}

// The four pairs of a key word (kv_layout.cuh) as 2u - 15: 1024 + 2u - 1039 and (1024 + 32u) / 16 - 79, both exact.
__device__ __forceinline__ void key_halves(uint32_t w, uint32_t* p) {
  const uint32_t r = __funnelshift_r(w, w, 8);
  const __half2 k1 = u32_h2(0xe40fe40fu), k16 = u32_h2(0x2c002c00u), k79 = u32_h2(0xd4f0d4f0u);  // -1039, 1/16, -79
  p[0] = h2_u32(__hadd2(code_bits(w, 0x001e001eu), k1));
  p[1] = h2_u32(__hfma2(code_bits(w, 0x01e001e0u), k16, k79));
  p[2] = h2_u32(__hadd2(code_bits(r, 0x001e001eu), k1));
  p[3] = h2_u32(__hfma2(code_bits(r, 0x01e001e0u), k16, k79));
}

// 2u - 15 for the codes at bits 1-4 of both halves, and at bits 5-8:
// 1024 + 2u - 1039 and (1024 + 32u) / 16 - 79.
__device__ __forceinline__ uint32_t value_low(uint32_t w) {
  return h2_u32(__hadd2(code_bits(w, 0x001e001eu), u32_h2(0xe40fe40fu)));
}
__device__ __forceinline__ uint32_t value_high(uint32_t w) {
  return h2_u32(__hfma2(code_bits(w, 0x01e001e0u), u32_h2(0x2c002c00u), u32_h2(0xd4f0d4f0u)));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(SFFN_FULL_MASK, v, 1);
  return v + __shfl_xor_sync(SFFN_FULL_MASK, v, 2);
}
// Over the eight lanes that share t.
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(SFFN_FULL_MASK, v, 4);
  v += __shfl_xor_sync(SFFN_FULL_MASK, v, 8);
  return v + __shfl_xor_sync(SFFN_FULL_MASK, v, 16);
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(SFFN_FULL_MASK, v, 4));
  v = fmaxf(v, __shfl_xor_sync(SFFN_FULL_MASK, v, 8));
  return fmaxf(v, __shfl_xor_sync(SFFN_FULL_MASK, v, 16));
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(SFFN_FULL_MASK, v, 1));
  return fmaxf(v, __shfl_xor_sync(SFFN_FULL_MASK, v, 2));
}

}  // namespace sffn
