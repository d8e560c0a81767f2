// act8_kernels.hip -- 8-bit activation checkpoints: rows packed to e4m3 codes with
// a power of two per block of 32, and back.
#include <algorithm>

#include "act8_device.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kHalf = kActBlock / 2;   // elements a thread moves

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Sixteen elements as they lie in memory: their largest magnitude's bits (as
// binary32), and their codes for a scale, four to a word.
template <typename T>
struct Half;
template <>
struct Half<uint16_t> {
    unsigned w[kHalf / 2];
    __device__ __forceinline__ void load(const uint16_t *p)
    {
        const u32x4 a = *reinterpret_cast<const u32x4_at2 *>(p), b = *reinterpret_cast<const u32x4_at2 *>(p + 8);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
    __device__ __forceinline__ void load(const uint16_t *p, int n)
    {
#pragma unroll
        for (int k = 0; k < kHalf / 2; ++k)
            w[k] = (2 * k < n ? p[2 * k] : 0u) | (2 * k + 1 < n ? (unsigned)p[2 * k + 1] << 16 : 0u);
    }
    __device__ __forceinline__ float at(int k) const { return k % 2 ? bf_hi(w[k / 2]) : bf_lo(w[k / 2]); }
    __device__ __forceinline__ unsigned top() const
    {
        u16x2 m = {0, 0};   // two at a time
#pragma unroll
        for (int k = 0; k < kHalf / 2; ++k)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[k] & 0x7fff7fffu));
        return (unsigned)max(m.x, m.y) << 16;
    }
    __device__ __forceinline__ unsigned codes(int k, float s) const
    {
        i16x2 c = {};
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2v, w[2 * k]), s, false);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2v, w[2 * k + 1]), s, true);
        return __builtin_bit_cast(unsigned, c);
    }
};
template <>
struct Half<float> {
    float x[kHalf];
    __device__ __forceinline__ void load(const float *p)
    {
#pragma unroll
        for (int i = 0; i < kHalf; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4_at4 *>(p + i);
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void load(const float *p, int n)
    {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            x[k] = k < n ? p[k] : 0.0f;
    }
    __device__ __forceinline__ float at(int k) const { return x[k]; }
    __device__ __forceinline__ unsigned top() const
    {
        unsigned m = 0;
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            m = max(m, __float_as_uint(x[k]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ unsigned codes(int k, float s) const
    {
        i16x2 c = {};
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[4 * k], x[4 * k + 1], s, false);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x[4 * k + 2], x[4 * k + 3], s, true);
        return __builtin_bit_cast(unsigned, c);
    }
};

constexpr unsigned kInfBits = 0x7f800000u;

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
    const T *p = static_cast<const T *>(a.x) + r * a.stride + c;
    Half<T> x;
    if (n >= kHalf)
        x.load(p);
    else
        x.load(p, n);
    unsigned top = x.top();
    const bool special = __any(top >= kInfBits);   // NaN or an infinity in the wave
    if (special) {
        top = 0;
#pragma unroll
        for (int k = 0; k < kHalf; ++k) {
            const unsigned b = __float_as_uint(x.at(k)) & 0x7fffffffu;
            top = max(top, b < kInfBits ? b : 0);
        }
    }
    top = max(top, (unsigned)__shfl_xor((int)top, 1, kWave));
    const unsigned byte = scale_byte(top);
    const float s = scale_of(byte);
    unsigned w[kHalf / 4];
#pragma unroll
    for (int k = 0; k < kHalf / 4; ++k)
        w[k] = x.codes(k, s);
    if (special) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            if ((__float_as_uint(x.at(k)) & 0x7fffffffu) >= kInfBits)
                w[k / 4] = (w[k / 4] & ~(0xffu << (8 * (k % 4)))) | 0x7fu << (8 * (k % 4));
    }
    uint8_t *q = a.codes + r * a.cols + c;
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

// A half block's values in memory.
__device__ __forceinline__ void put_values(uint16_t *p, int n, const unsigned (&w)[kHalf / 4], float s)
{
    unsigned v[kHalf / 2];
#pragma unroll
    for (int k = 0; k < kHalf / 4; ++k) {
        v[2 * k] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[k], s, false));
        v[2 * k + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[k], s, true));
    }
    if (n >= kHalf) {
        *reinterpret_cast<u32x4_at2 *>(p) = u32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<u32x4_at2 *>(p + 8) = u32x4{v[4], v[5], v[6], v[7]};
        return;
    }
#pragma unroll
    for (int k = 0; k < kHalf; ++k)
        if (k < n)
            p[k] = (uint16_t)(v[k / 2] >> (16 * (k % 2)));
}
__device__ __forceinline__ void put_values(float *p, int n, const unsigned (&w)[kHalf / 4], float s)
{
    float x[kHalf];
#pragma unroll
    for (int k = 0; k < kHalf / 4; ++k)
        widen_codes(w[k], s, x + 4 * k);
    store_n(p, n, reinterpret_cast<float (&)[kOct]>(x[0]));
    store_n(p + kOct, n - kOct, reinterpret_cast<float (&)[kOct]>(x[kOct]));
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
    if (n >= kHalf) {
        const u32x4 v = *reinterpret_cast<const u32x4_at1 *>(q);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < kHalf; ++k)
            if (k < n)
                w[k / 4] |= (unsigned)q[k] << (8 * (k % 4));
    }
    put_values(static_cast<T *>(a.x) + r * a.stride + c, n, w, s);
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
