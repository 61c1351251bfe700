// Device helpers of the 8-bit checkpoints (gfx950): E4M3 codes with one power-of-two scale
// per 32 neighbours of a row, stored as the biased exponent of the scale.
#pragma once

#include "common.h"

namespace moe {

constexpr int kCkptBlock = 32;
constexpr int kCkptMinExp = 10;  // biased: 2^-117, so that the smallest code (2^-9) stays a normal bf16

MOE_DEV float ckpt_scale(uint32_t biased) { return __uint_as_float(biased << 23); }

// 8 codes (two words) -> 8 bf16, exact: the conversion applies the scale's exponent
MOE_DEV u32x4_t ckpt_to_bf16(u32x2_t w, float scale) {
  return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[0], scale, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[0], scale, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[1], scale, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[1], scale, true))};
}

}  // namespace moe
