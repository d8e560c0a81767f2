// act8_kernels.hip -- 8-bit activation checkpoints: rows packed to e4m3 codes with
// a power of two per block of 32, and back.
#include <algorithm>

#include "act8_device.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kHalf = kActBlock / 2;   // elements a thread moves

// A finite magnitude's bits; 0 for NaN and infinities.
__device__ __forceinline__ unsigned magnitude(float x)
{
    const unsigned b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0;
}

// The scale's byte for a block whose largest magnitude has these bits: 448 =
// 1.75 * 2^8, so the exponent - 8, one more where the mantissa exceeds 1.75.
__device__ __forceinline__ unsigned scale_byte(unsigned top)
{
    return (unsigned)max((int)((top + 0x1fffffu) >> 23) - 8, 0);
}

// One thread per half block; the two of a block are neighbours in a wave.
template <typename T>
__global__ __launch_bounds__(kBlock) void pack_kernel(Act8Args a, int64_t row0, uint32_t halves, uint32_t total)
{
    const uint32_t i = blockIdx.x * kBlock + threadIdx.x;
    if (i >= total)
        return;
    const int64_t r = row0 + i / halves;
    const int h = (int)(i % halves), c = h * kHalf, n = min(a.cols - c, kHalf);
    float x[kHalf];
    const T *p = static_cast<const T *>(a.x) + r * a.stride + c;
    load_n(p, n, reinterpret_cast<float (&)[kOct]>(x[0]));
    load_n(p + kOct, n - kOct, reinterpret_cast<float (&)[kOct]>(x[kOct]));
    unsigned top = 0;
#pragma unroll
    for (int k = 0; k < kHalf; ++k)
        top = max(top, magnitude(x[k]));
    top = max(top, (unsigned)__shfl_xor((int)top, 1, kWave));
    const unsigned byte = scale_byte(top);
    const float inv = __uint_as_float((254 - byte) << 23);   // 2^(127 - byte)
    unsigned w[kHalf / 4];
#pragma unroll
    for (int k = 0; k < kHalf; ++k)   // an infinity as NaN: the codes have none
        x[k] = __builtin_fabsf(x[k]) == __builtin_inff() ? __builtin_nanf("") : x[k] * inv;
#pragma unroll
    for (int k = 0; k < kHalf / 4; ++k) {
        w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k], x[4 * k + 1], 0, false);
        w[k] = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * k + 2], x[4 * k + 3], w[k], true);
    }
    uint8_t *q = a.codes + r * a.cols + c;
    typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
    if (n >= kHalf)
        *reinterpret_cast<u32x4_at1 *>(q) = u32x4{w[0], w[1], w[2], w[3]};
    else
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            if (k < n)
                q[k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
    if (h % 2 == 0)
        a.scales[r * a.blocks + h / 2] = (uint8_t)byte;
}

template <typename T>
__global__ __launch_bounds__(kBlock) void unpack_kernel(Act8Args a, int64_t row0, uint32_t halves, uint32_t total)
{
    const uint32_t i = blockIdx.x * kBlock + threadIdx.x;
    if (i >= total)
        return;
    const int64_t r = row0 + i / halves;
    const int h = (int)(i % halves), c = h * kHalf, n = min(a.cols - c, kHalf);
    if (n <= 0)
        return;
    const uint8_t *q = a.codes + r * a.cols + c;
    const float s = scale_of(a.scales[r * a.blocks + h / 2]);
    unsigned w[kHalf / 4] = {};
    typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
    if (n >= kHalf) {
        const u32x4 v = *reinterpret_cast<const u32x4_at1 *>(q);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            if (k < n)
                w[k / 4] |= (unsigned)q[k] << (8 * (k % 4));
    }
    float x[kHalf];
#pragma unroll
    for (int k = 0; k < kHalf / 4; ++k)
        widen_codes(w[k], s, x + 4 * k);
    T *p = static_cast<T *>(a.x) + r * a.stride + c;
    store_n(p, n, reinterpret_cast<float (&)[kOct]>(x[0]));
    store_n(p + kOct, n - kOct, reinterpret_cast<float (&)[kOct]>(x[kOct]));
}

// f(first row, half blocks of a row, half blocks of the launch) for launches whose
// threads 32 bits count.
template <typename F>
void each_launch(const Act8Args &a, F f)
{
    const uint32_t halves = 2 * (uint32_t)a.blocks;
    const int64_t most = (int64_t(1) << 31) / halves;
    for (int64_t r = 0; r < a.rows; r += most)
        f(r, halves, (uint32_t)(std::min(most, a.rows - r) * halves));
}

}  // namespace

int launch_act8_pack(const Act8Args &a, void *stream)
{
    each_launch(a, [&](int64_t r, uint32_t halves, uint32_t total) {
        const dim3 grid((total + kBlock - 1) / kBlock);
        if (a.dtype == ZERO_F32)
            hipLaunchKernelGGL((pack_kernel<float>), grid, dim3(kBlock), 0, reinterpret_cast<hipStream_t>(stream), a,
                               r, halves, total);
        else
            hipLaunchKernelGGL((pack_kernel<uint16_t>), grid, dim3(kBlock), 0, reinterpret_cast<hipStream_t>(stream),
                               a, r, halves, total);
    });
    return hipGetLastError();
}

int launch_act8_unpack(const Act8Args &a, void *stream)
{
    each_launch(a, [&](int64_t r, uint32_t halves, uint32_t total) {
        const dim3 grid((total + kBlock - 1) / kBlock);
        if (a.dtype == ZERO_F32)
            hipLaunchKernelGGL((unpack_kernel<float>), grid, dim3(kBlock), 0, reinterpret_cast<hipStream_t>(stream),
                               a, r, halves, total);
        else
            hipLaunchKernelGGL((unpack_kernel<uint16_t>), grid, dim3(kBlock), 0,
                               reinterpret_cast<hipStream_t>(stream), a, r, halves, total);
    });
    return hipGetLastError();
}

}  // namespace zero
