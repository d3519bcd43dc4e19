// The scale and the codes of a block of 128 values quantized to E4M3, shared by the quantizers.
//
// A block's scale is d = amax / 448, its codes E4M3(v * (448 / amax)) rounded to nearest even, so the
// largest magnitude takes the largest code.  Both quotients are fp32 divisions rounded to nearest and
// kept to normal numbers (d >= 2^-126, factor <= 2^126: a smaller amax uses fewer of the codes); a
// block of zeros has d = 1.  The amax is taken on the bit patterns, whose order is that of the
// magnitudes with infinity and NaN on top: a block that holds either gets a scale that makes all of
// its values infinite or NaN instead of hiding them.
#pragma once
#include "common.h"

namespace moe {

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The maximum over each 16 lanes: DPP moves (lanes ^ 1, lanes ^ 2, mirrors of 8 and of 16).
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = umax(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));
  m = umax(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));
  m = umax(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));
  return umax(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, true));
}

struct BlockScale {
  float factor, d;
};
// amax as bits of a non-negative float
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  const float amax = __builtin_bit_cast(float, amax_bits);
  if (amax_bits == 0) return {1.0f, 1.0f};
  const float f = 448.0f / amax, d = amax / 448.0f;
  return {f > 0x1p126f ? 0x1p126f : f, d < 0x1p-126f ? 0x1p-126f : d};   // (a NaN passes)
}

// codes of a and b times f in the low (hi == false) or high half of old.  |v f| <= 448 (1 + 2^-22),
// which rounds to 448, so nothing has to be clamped.
template <bool hi>
__device__ __forceinline__ uint32_t codes2(float a, float b, float f, uint32_t old) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a * f, b * f, (int)old, hi);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float f) {
  return codes2<true>(c, d, f, codes2<false>(a, b, f, 0u));
}

}  // namespace moe
