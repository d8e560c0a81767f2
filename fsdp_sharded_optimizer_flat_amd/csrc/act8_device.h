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

// The first m of four neighbouring elements of d_w: written, or added to what is there.
template <typename O>
__device__ __forceinline__ void put4(O *p, int m, const float (&v)[4], int accumulate)
{
    typedef O Four __attribute__((ext_vector_type(4)));
    typedef Four Four_at __attribute__((aligned(sizeof(O))));
    float x[4] = {v[0], v[1], v[2], v[3]};
    if (m >= 4) {
        if (accumulate) {
            const Four was = *reinterpret_cast<const Four_at *>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[k] = widen<O>(was[k]) + v[k];
        }
        Four now;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            now[k] = narrow<O>(x[k]);
        *reinterpret_cast<Four_at *>(p) = now;
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < m)
            p[k] = narrow<O>(accumulate ? widen<O>(p[k]) + v[k] : v[k]);
}

}  // namespace dev
}  // namespace zero
