// What token_loss_device.h and device_common.h use of HIP and of gfx950's
// builtins, for one thread at a time on the CPU: found before the real header
// where a test compiles the device code for the host.  Buffer accesses keep the
// hardware's range check: what lies outside a buffer reads as zero and is not
// stored.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#define __device__
#define __host__
#define __global__
#define __shared__ static
#define __forceinline__ inline
#define asm                 // the device code's barriers are `asm volatile(...)`
#define volatile(...)

struct Dim3 {
    unsigned x, y, z;
};
inline Dim3 threadIdx, blockIdx, blockDim, gridDim;

typedef void *hipStream_t;
typedef int hipError_t;
constexpr hipError_t hipSuccess = 0;
inline hipError_t hipGetLastError() { return hipSuccess; }

inline int max(int a, int b) { return a > b ? a : b; }
inline int min(int a, int b) { return a < b ? a : b; }
inline float __uint_as_float(unsigned x) { return __builtin_bit_cast(float, x); }
inline unsigned __float_as_uint(float x) { return __builtin_bit_cast(unsigned, x); }
inline float __int_as_float(int x) { return __builtin_bit_cast(float, x); }
inline int __float_as_int(float x) { return __builtin_bit_cast(int, x); }
inline void __syncthreads() {}
inline bool __any(bool x) { return x; }
template <typename T>
inline T __shfl_xor(T x, int, int) { return x; }

struct HostBuffer {
    char *p;
    int64_t bytes;
};
typedef unsigned int host_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int host_u32x2 __attribute__((ext_vector_type(2)));
template <typename V>
inline V host_buffer_load(const HostBuffer &b, int at, int first)
{
    V v{};
    const int64_t o = (int64_t)(uint32_t)at + (uint32_t)first;
    if (o + (int64_t)sizeof(V) <= b.bytes)
        std::memcpy(&v, b.p + o, sizeof(V));
    return v;
}
template <typename V>
inline void host_buffer_store(V v, const HostBuffer &b, int at, int first)
{
    const int64_t o = (int64_t)(uint32_t)at + (uint32_t)first;
    if (o + (int64_t)sizeof(V) <= b.bytes)
        std::memcpy(b.p + o, &v, sizeof(V));
}
template <typename T>
inline HostBuffer host_buffer(const T *p, int bytes)
{
    return {const_cast<char *>(reinterpret_cast<const char *>(p)), bytes};
}
#define __amdgpu_buffer_rsrc_t HostBuffer
#define __builtin_amdgcn_make_buffer_rsrc(p, stride, bytes, flags) host_buffer(p, bytes)
#define __builtin_amdgcn_raw_buffer_load_b128(b, at, first, policy) host_buffer_load<host_u32x4>(b, at, first)
#define __builtin_amdgcn_raw_buffer_load_b64(b, at, first, policy) host_buffer_load<host_u32x2>(b, at, first)
#define __builtin_amdgcn_raw_buffer_store_b128(v, b, at, first, policy) host_buffer_store(v, b, at, first)
#define __builtin_amdgcn_raw_buffer_store_b64(v, b, at, first, policy) host_buffer_store(v, b, at, first)
#define __builtin_amdgcn_readfirstlane(x) (x)
#define __builtin_amdgcn_readlane(x, lane) (x)
#define __builtin_amdgcn_update_dpp(old, x, ctrl, rows, banks, bound) (x)
#define __builtin_amdgcn_exp2f(x) std::exp2(x)
#define __builtin_amdgcn_sched_barrier(mask) ((void)0)
