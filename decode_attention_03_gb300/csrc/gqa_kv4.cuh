// The 4-bit cache (kv4): its layout, and the conversions in both directions.
//
// A (block, head) is one contiguous stretch of block_size * (D + D/8) bytes (a multiple of 16): K codes, V codes, K scales,
// V scales.  A code is sign and e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6), two in a byte; every 16 elements of a row have a scale
// byte, the upper byte of a binary16 number (e5m2 without a sign), so that one byte permutation makes scales of any two
// groups a pair of f16, and a code times its scale (2 + 3 significant bits) is exact in f16 and in bfloat16.
// The 16-byte chunks of a row are stored where the bank swizzle wants them: a bulk copy of a whole (block, head) lands
// ready for conflict-free transposing ldmatrix (V) and for 16-byte reads (K: chunk c of a row is what lane c of a
// row's four holds of the MMA's A operand, two whole groups).
// Error of a row of normal values, relative to its size: 0.098 (scales with 3 bits behind the leading one instead of 2: 0.095,
// with none 0.113; a scale for each row instead of each 16 would be 0.12 or more).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "ptx.cuh"

namespace gqa {

constexpr float kKv4MaxScale = 10240.f;     // 6 times this is the largest value: binary16 holds it
constexpr uint32_t kKv4NanScale = 0x7f;     // scale byte of 16 elements with a NaN or an infinity among them
constexpr uint32_t kKv4Infinite = 0x7c;     // scale bytes from here on are not finite (those above 0x71 = 10240 are not written)

__host__ __device__ constexpr int kv4_block_bytes(int block_size, int D) { return block_size * (D + D / 8); }

// byte offset, among a (block, head)'s K or V codes, of 16-byte chunk c of row r
template <int D>
__host__ __device__ constexpr int kv4_chunk(int r, int c) {
  return r * (D / 2) + ((c ^ (D == 128 ? ((r >> 1) & 3) : ((r >> 2) & 1))) << 4);
}

// x / s in fp32, rounded to nearest, where inv is the fp32 number nearest to 1 / s and nothing overflows: a product and one
// correction by its exact remainder (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  A value on the border of two codes must come out there: x * inv alone misses it for s = 1.75 * 2^k.
__device__ __forceinline__ float kv4_quotient(float x, float s, float inv) {
  const float q = x * inv;
  return fmaf(fmaf(-q, s, x), inv, q);
}

// scale byte of 16 elements whose largest magnitude has the bits `top`: m / 6 rounded to nearest even
__device__ __forceinline__ uint32_t kv4_scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return kKv4NanScale;
  const float s = fminf(kv4_quotient(__uint_as_float(top), 6.f, 1.f / 6.f), kKv4MaxScale);
  uint16_t two;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(s));
  return two & 0xffu;
}

__device__ __forceinline__ float kv4_scale(uint32_t byte) {
  float f;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(byte << 8));
  return f;
}

// the fp32 number nearest to 1 / s of a scale s > 0: one of four significands
__device__ __forceinline__ float kv4_inverse(float s) {
  const uint32_t b = __float_as_uint(s);
  const float f = b & 0x400000u ? (b & 0x200000u ? 4.f / 7.f : 2.f / 3.f) : (b & 0x200000u ? 0.8f : 1.f);
  return __uint_as_float(__float_as_uint(f) + 0x3f800000u - (b & 0x7f800000u));
}

// codes of x[0..3] / s in the low 16 bits, nearest even, beyond 6 saturated; inv: kv4_inverse(s).  (Codes below a scale that
// is not finite are no values.)
__device__ __forceinline__ uint32_t kv4_codes(const float* x, float s, float inv) {
  float z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = kv4_quotient(x[i], s, inv);
  uint32_t r;
  asm("{\n\t.reg .b8 a, b;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b, a, b};\n\t}"
      : "=r"(r) : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
  return r & 0xffffu;
}

// the eight codes of a word as four pairs of f16, a byte each
__device__ __forceinline__ void kv4_unpack(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// two scales as a pair of f16: `pick` names a byte of a, b for each, kv4_pick(i, j) for byte i of a and j of b
__device__ __forceinline__ uint32_t kv4_pick(uint32_t i, uint32_t j) {
  return (8 + i) | (i << 4) | ((12 + j) << 8) | ((4 + j) << 12);   // (8 + i: the sign of byte i, which is 0, eight times)
}
__device__ __forceinline__ uint32_t kv4_scales(uint32_t a, uint32_t b, uint32_t pick) {
  uint32_t h;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(h) : "r"(a), "r"(b), "r"(pick));
  return h;
}

__device__ __forceinline__ uint32_t kv4_mul(uint32_t x, uint32_t s) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(s));
  return y;
}

}  // namespace gqa
