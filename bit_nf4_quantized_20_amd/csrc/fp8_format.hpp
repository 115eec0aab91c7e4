// fp8_format.hpp -- the 8-bit block-scaled format: e4m3 codes (OCP: bias 7,
// largest finite 448, no infinities) with one power-of-two scale per block,
// stored as its biased exponent (byte b = 2^(b - 127)).
//
// For a block whose largest magnitude is a, the scale is 2^e with e the least
// integer such that a 2^-e <= 448 = 1.75 2^8.  Writing a = m 2^p, 1 <= m < 2,
// that is e = p - 8 for m <= 1.75 and p - 7 above; it comes from a's bits with
// one integer addition (adding 2^23 - 1 - (0.75 2^23) carries into the
// exponent exactly when m > 1.75).  e is held to >= -127; an all-zero block
// has byte 0.  Because the scale is a power of two, w 2^-e and code 2^e are
// exact in fp32, so a code is one rounding of the weight, and
// v_mfma_scale applies the scales inside the matrix cores at no cost.  The
// price against a free fp32 scale is at most one bit of the block's range at
// its bottom end (the largest code lies in (224, 448] instead of at 448); the
// codes' relative precision is the same.
#pragma once

#include "common.hpp"

namespace qlora {

constexpr int kF8Block = 128;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// scale byte of a block whose largest |value| has the fp32 bits a (a finite)
__host__ __device__ constexpr uint32_t f8_scale_byte(uint32_t a) {
  // exponent field of a (p + 127), plus 1 where the fraction exceeds 0.75
  const int e = static_cast<int>((a + 0x1fffffu) >> 23) - 8;
  return static_cast<uint32_t>(e > 0 ? e : 0);
}
static_assert(f8_scale_byte(0x43e00000u) == 127, "448 -> 2^0");
static_assert(f8_scale_byte(0x43e00001u) == 128, "above 448 -> 2^1");
static_assert(f8_scale_byte(0x43600000u) == 126 && f8_scale_byte(0) == 0, "224 -> 2^-1, 0 -> byte 0");

// 2^(b - 127) and 2^(127 - b) as fp32 for a scale byte b <= 248
__device__ __forceinline__ float f8_scale(uint32_t b) {
  return __builtin_bit_cast(float, b == 0 ? 0x00400000u : b << 23);
}
__device__ __forceinline__ float f8_inv_scale(uint32_t b) { return __builtin_bit_cast(float, (254u - b) << 23); }

// four fp32 -> four e4m3 codes (round to nearest even)
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return static_cast<uint32_t>(v);
}

}  // namespace qlora
