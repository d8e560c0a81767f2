// act8_device.h -- the format of the 8-bit activation checkpoints on the device.
#pragma once

#include "act8.h"
#include "octs.h"

namespace zero {
namespace dev {

// 2^(byte - 127); 255 marks a block of NaN.
__device__ __forceinline__ float scale_of(unsigned byte)
{
    const float s = __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
    return byte == 255 ? __builtin_nanf("") : s;
}

// Four codes (a word, lowest byte first) times a scale.
__device__ __forceinline__ void widen_codes(unsigned w, float s, float *x)
{
    const f32x2 lo = __builtin_bit_cast(f32x2, __builtin_amdgcn_cvt_pk_f32_fp8(w, false));
    const f32x2 hi = __builtin_bit_cast(f32x2, __builtin_amdgcn_cvt_pk_f32_fp8(w, true));
    x[0] = lo.x * s, x[1] = lo.y * s, x[2] = hi.x * s, x[3] = hi.y * s;
}

}  // namespace dev
}  // namespace zero
