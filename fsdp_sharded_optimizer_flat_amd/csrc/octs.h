// octs.h -- eight consecutive elements of a row, binary32 or bf16, at any element's
// address, for the kernels over rows of any width and stride.
#pragma once

#include "device_common.h"

namespace zero {
namespace dev {

typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t x) { return __uint_as_float((unsigned)x << 16); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float x) { return to_bf16(x); }

// Eight consecutive elements at any element's address.
__device__ __forceinline__ void load8(const uint16_t *p, float (&x)[kOct])
{
    const u32x4 r = *reinterpret_cast<const u32x4_at2 *>(p);
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[2 * i] = bf_lo(w[i]), x[2 * i + 1] = bf_hi(w[i]);
}
__device__ __forceinline__ void load8(const float *p, float (&x)[kOct])
{
    const f32x4 a = *reinterpret_cast<const f32x4_at4 *>(p), b = *reinterpret_cast<const f32x4_at4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&x)[kOct])
{
    *reinterpret_cast<u32x4_at2 *>(p) = u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
}
__device__ __forceinline__ void store8(float *p, const float (&x)[kOct])
{
    *reinterpret_cast<f32x4_at4 *>(p) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4_at4 *>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
// Eight elements as they lie in memory.
template <typename T>
struct RawOct;
template <>
struct RawOct<uint16_t> {
    u32x4 a;
    __device__ __forceinline__ void load(const uint16_t *p) { a = *reinterpret_cast<const u32x4_at2 *>(p); }
    __device__ __forceinline__ void stream(const uint16_t *p)   // not read again soon
    {
        a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_at2 *>(p));
    }
    __device__ __forceinline__ void load(const uint16_t *p, int n)   // the first n
    {
#pragma unroll
        for (int k = 0; k < kOct / 2; ++k)
            a[k] = (2 * k < n ? p[2 * k] : 0u) | (2 * k + 1 < n ? (unsigned)p[2 * k + 1] << 16 : 0u);
    }
    __device__ __forceinline__ float at(int k) const { return k % 2 ? bf_hi(a[k / 2]) : bf_lo(a[k / 2]); }
};
template <>
struct RawOct<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const f32x4_at4 *>(p), b = *reinterpret_cast<const f32x4_at4 *>(p + 4);
    }
    __device__ __forceinline__ void stream(const float *p)
    {
        a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_at4 *>(p));
        b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_at4 *>(p + 4));
    }
    __device__ __forceinline__ void load(const float *p, int n)
    {
#pragma unroll
        for (int k = 0; k < kOct; ++k)
            if (k < 4)
                a[k] = k < n ? p[k] : 0.0f;
            else
                b[k - 4] = k < n ? p[k] : 0.0f;
    }
    __device__ __forceinline__ float at(int k) const { return k < 4 ? a[k] : b[k - 4]; }
};

// The first n of them (all eight, or the end of a row).
template <typename T>
__device__ __forceinline__ void load_n(const T *p, int n, float (&x)[kOct])
{
    if (n >= kOct) {
        load8(p, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < kOct; ++i)
        x[i] = i < n ? widen<T>(p[i]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_n(T *p, int n, const float (&x)[kOct])
{
    if (n >= kOct) {
        store8(p, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < kOct; ++i)
        if (i < n)
            p[i] = narrow<T>(x[i]);
}

}  // namespace dev

// f(element of the first type, of the second) for two dtypes.
template <typename F>
inline void by_types(int32_t d, int32_t o, F f)
{
    const float w = 0.0f;
    const uint16_t h = 0;
    if (d == ZERO_F32)
        o == ZERO_F32 ? f(w, w) : f(w, h);
    else
        o == ZERO_F32 ? f(h, w) : f(h, h);
}

}  // namespace zero
