// Device helpers of the microscaled 4-bit format (MXFP4), shared by its
// storage and product kernels.
//
// A row is cut into blocks of 32 values.  A block holds 32 e2m1 codes (sign,
// two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one
// scale byte s standing for 2^(s - 127); s = 255 makes the block NaN.  A value
// is code * 2^(s - 127).  Codes lie two to a byte, the even column in the low
// nibble, so a block is 16 bytes and is one lane's operand of the scaled
// matrix instructions.
#pragma once

#include "common.h"

namespace moe {

constexpr int kMxBlock = 32;       // values per scale
constexpr int kMxBlockBytes = 16;  // code bytes per block
constexpr int kMxNan = 255;        // scale byte of a block that holds a NaN or an infinity

// Scale byte of a block from the bits of its largest magnitude (an integer
// maximum of the absolute values' bits, in which every NaN is above infinity
// and infinity above the finite values): 2^(floor(log2 amax) - 2), which
// brings amax into [4, 8), the binade of the largest code.  The exponent
// field is floor(log2 amax) + 127, or 0 for zero and subnormals; below 2^-127
// the scale stays at 2^-127.
__device__ __forceinline__ int mx4_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  return e == 255 ? kMxNan : max(e - 2, 0);
}

// 1 / scale as a float: 2^(127 - s), between 2^-125 and 2^127, always normal.
// A NaN block gives 0.
__device__ __forceinline__ float mx4_inv_scale(int s) {
  return s == kMxNan ? 0.f : __uint_as_float((uint32_t)(254 - s) << 23);
}

__device__ __forceinline__ uint32_t f32_abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Eight values of one block to eight codes.  v * inv is exact (a power of two,
// the result below 8 and, for a subnormal v, normal), and the conversion
// rounds to the nearest code, ties to the even one, and holds magnitudes above
// 6 at 6: one rounding in all.  In a NaN block (inv = 0) every code is +0.
__device__ __forceinline__ uint32_t mx4_pack8(const float v[8], float inv) {
  uint32_t d = 0;
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[0] * inv, v[1] * inv, 1.0f, 0);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2] * inv, v[3] * inv, 1.0f, 1);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4] * inv, v[5] * inv, 1.0f, 2);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6] * inv, v[7] * inv, 1.0f, 3);
  return inv != 0.f ? d : 0u;
}

// Maximum over the four lanes of a quad, in every lane of it.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// The scale as the float operand of the conversion instructions, which read
// its exponent field alone (0 = 2^-127, 255 = NaN).
__device__ __forceinline__ float mx4_scale_f32(uint32_t s) { return __uint_as_float(s << 23); }

// Eight codes (one dword) to eight bf16 values, exactly: a code has two
// significant bits and the smallest magnitude, 2^-128, is a bf16 subnormal.
__device__ __forceinline__ uint4 mx4_unpack8_bf16(uint32_t d, float scale) {
  uint4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3));
  return o;
}

// float -> bf16 bits, to nearest even, NaN kept (f32_to_bf16_rne takes finite values only).
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

}  // namespace moe
