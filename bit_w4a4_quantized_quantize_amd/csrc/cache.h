// Device-side helpers shared by the kernels of the e4m3 cache (cache.hip, attention_cache.hip).
#pragma once

#include "common.h"
#include "kernels.h"

namespace svdq {

// 2^(b - 127) of an E8M0 byte in the form the scaled conversions take (they read the exponent field); 255 is NaN
__device__ __forceinline__ float cache_scale(uint32_t b) { return __uint_as_float(b < 255u ? b << 23 : 0x7FC00000u); }

// Codes 2 HALF, 2 HALF + 1 of a dword times the scale's power of two, as two bf16 (exact: an e4m3 value has four
// significant bits)
template <int HALF>
__device__ __forceinline__ uint32_t fp8_pair_to_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HALF != 0));
}

}  // namespace svdq
