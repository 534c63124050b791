// Device helpers of the microscaled format (include/i4s_prompt.h), gfx950.
#pragma once

#include "i4s_gemv_common.h"
#include "i4s_prompt_internal.h"

namespace i4s {
namespace {

typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

// 16-bit activation types: the largest magnitude as bits, and eight values as
// 4-bit codes.  v_cvt_scalef32_pk_fp4 divides by a power of two, rounds to
// nearest even and saturates.
struct HalfX {
  static __device__ float to_float(uint32_t bits) { return fp16_bits_to_float(bits); }
  static constexpr uint32_t kInf = 0x7C00u;
  template <int B>
  static __device__ uint32_t code(uint32_t old, uint32_t w, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(h2_t, w), scale, B);
  }
};
struct BrainX {
  static __device__ float to_float(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }
  static constexpr uint32_t kInf = 0x7F80u;
  template <int B>
  static __device__ uint32_t code(uint32_t old, uint32_t w, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(b2_t, w), scale, B);
  }
};

// Larger of the 16-bit halves.
__device__ inline uint32_t max_halves(uint32_t a, uint32_t b) {
  typedef uint16_t us2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}

// Magnitude bits of eight values: the larger of even and of odd ones.
__device__ inline uint32_t top_bits(u4_t v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return max_halves(max_halves(v.x & kAbs, v.y & kAbs), max_halves(v.z & kAbs, v.w & kAbs));
}

// Largest of the four lanes of a quad.
__device__ inline uint32_t quad_max(uint32_t v) {
  v = max_halves(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false));  // lanes 1 0 3 2
  return max_halves(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false));  // lanes 2 3 0 1
}

// A block's scale byte from the bits of its largest magnitude (their order is
// that of the values; a NaN lies above infinity).
template <typename X>
__device__ inline uint32_t scale_byte(uint32_t top) {
  const uint32_t f = __builtin_bit_cast(uint32_t, X::to_float(top));
  const uint32_t e = f >> 23;  // 0 for 0 and below 2^-126
  return top >= X::kInf ? kMxNaN : (e > 2 ? e - 2 : 0);
}
// Its power of two, as the conversion takes it (2^-127 has no exponent bits).
__device__ inline float scale_value(uint32_t byte) {
  return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

// Eight values as eight codes.
template <typename X>
__device__ inline uint32_t codes(u4_t v, float scale) {
  uint32_t r = X::template code<0>(0u, v.x, scale);
  r = X::template code<1>(r, v.y, scale);
  r = X::template code<2>(r, v.z, scale);
  return X::template code<3>(r, v.w, scale);
}

}  // namespace
}  // namespace i4s
