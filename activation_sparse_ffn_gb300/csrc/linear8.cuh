// Where the codes of the 8-bit linear layer stand, and how they become
// half-precision numbers.
//
// Codes are packed once into blocks of 128 rows x 64 inputs, a row's 64 bytes
// beside each other: [tile of 128 rows][64 inputs][row][64 bytes], 8 KB a block.
// A code c is stored as c + 128. The 16-byte chunk with inputs 16 t .. 16 t + 15
// of row r stands at chunk position t ^ ((r >> 1) & 3), so that eight
// consecutive rows' chunks t lie in different banks of shared memory.
//
// GB300 has no 8-bit whole-number form of its tensor instructions
// (kind::i8 is not offered for sm_103a, and the warp-level form issues at 257
// multiply-adds per SM and cycle, a quarter of the half-precision form's 1011, both measured). A code is a half
// exactly, a product of two codes at most 2^14, and a sum of 1024 of them at
// most 2^24, which an fp32 accumulator holds exactly: sums leave it as whole
// numbers every 1024 inputs at the latest.
#pragma once

#include "common.cuh"

namespace sffn {

constexpr int kL8Rows = 128, kL8Inputs = 64, kL8Block = kL8Rows * kL8Inputs;   // a packed block
constexpr int kL8Exact = 1024;                                                // inputs that an fp32 sum is exact for

// Byte offset of chunk t (16 inputs) of row r in its block.
__host__ __device__ constexpr int l8_chunk(int r, int t) { return r * 64 + ((t ^ ((r >> 1) & 3)) << 4); }

// Four stored codes as four halves: u in the low byte of a half whose exponent is that of 1024 is 1024 + u exactly, and
// 1024 + 128 taken off leaves c.
__device__ __forceinline__ void l8_halves(uint32_t u, uint32_t& lo, uint32_t& hi) {
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&a), off), q = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&p), hi = *reinterpret_cast<const uint32_t*>(&q);
}

// The output of one row and token from its exact sum, one rounding per operation.
__device__ __forceinline__ float l8_value(int sum, float scale, float x_scale, float bias) {
  return __fadd_rn(__fmul_rn(__int2float_rn(sum), __fmul_rn(scale, x_scale)), bias);
}

}  // namespace sffn
