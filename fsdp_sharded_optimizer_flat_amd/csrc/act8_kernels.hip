// act8_kernels.hip -- 8-bit activation checkpoints: rows packed to e4m3 codes with
// a power of two per block of 32, and back.
#include <algorithm>

#include "act8_device.h"

namespace zero {
namespace {

using namespace dev;

// Bound by memory.  Four neighbouring lanes share a block, eight elements each; a
// thread takes kTurns of them, so that its loads wait together, streamed past the
// caches (8192 x 14336 bf16 there and back: 116 us, 6.1 TB/s; 132 with sixteen
// elements to a thread and ordinary loads and stores).
constexpr int kLanes = kActBlock / kOct, kTurns = 2;

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));

// The largest magnitude's bits, as binary32.
__device__ __forceinline__ unsigned top_of(const RawOct<uint16_t> &x)
{
    u16x2 m = {0, 0};   // two elements at a time
#pragma unroll
    for (int k = 0; k < 4; ++k)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x.a[k] & 0x7fff7fffu));
    return (unsigned)max(m.x, m.y) << 16;
}
__device__ __forceinline__ unsigned top_of(const RawOct<float> &x)
{
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < kOct; ++k)
        m = max(m, __float_as_uint(x.at(k)) & 0x7fffffffu);
    return m;
}
// Elements 4 i .. 4 i + 3 over s, rounded to codes, lowest byte first.
__device__ __forceinline__ unsigned codes_of(const RawOct<uint16_t> &x, int i, float s)
{
    const unsigned lo = x.a[2 * i], hi = x.a[2 * i + 1];   // (bit_cast of an element takes the vector's first)
    i16x2 c = {};
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2v, lo), s, false);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(c, __builtin_bit_cast(bf16x2v, hi), s, true);
    return __builtin_bit_cast(unsigned, c);
}
__device__ __forceinline__ unsigned codes_of(const RawOct<float> &x, int i, float s)
{
    i16x2 c = {};
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x.at(4 * i), x.at(4 * i + 1), s, false);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(c, x.at(4 * i + 2), x.at(4 * i + 3), s, true);
    return __builtin_bit_cast(unsigned, c);
}

constexpr unsigned kInfBits = 0x7f800000u;

// The scale's byte for a block whose largest magnitude has these bits: 448 =
// 1.75 * 2^8, so the exponent - 8, one more where the mantissa exceeds 1.75.
__device__ __forceinline__ unsigned scale_byte(unsigned top)
{
    return (unsigned)max((int)((top + 0x1fffffu) >> 23) - 8, 0);
}

// The largest of a block's lanes (neighbours: quads of a wave), in each.
__device__ __forceinline__ unsigned block_max(unsigned x)
{
    x = max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0xb1, 0xf, 0xf, false));   // lane ^ 1
    return max(x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, 0x4e, 0xf, 0xf, false));   // lane ^ 2
}

// The piece of a row that a thread takes in a turn: row r, n <= 8 elements (none, past a
// row's end in its last block) from column c on.
struct Piece8 {
    int64_t r;
    int lane, c, n;
    __device__ __forceinline__ Piece8(const Act8Args &a, int64_t row0, uint32_t i)
    {
        const uint32_t per_row = (uint32_t)a.blocks * kLanes;
        r = row0 + i / per_row;
        lane = (int)(i % per_row);
        c = lane * kOct;
        n = min(a.cols - c, kOct);
    }
};

template <typename T>
__global__ __launch_bounds__(kBlock) void pack_kernel(Act8Args a, int64_t row0, uint32_t total)
{
    const uint32_t i0 = blockIdx.x * (kBlock * kTurns) + threadIdx.x;
    RawOct<T> x[kTurns];
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        const Piece8 p(a, row0, min(i0 + u * kBlock, total - 1));
        const T *from = static_cast<const T *>(a.x) + p.r * a.stride + p.c;
        if (p.n >= kOct)
            x[u].stream(from);
        else
            x[u].load(from, p.n);
    }
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        if (i0 + u * kBlock >= total)   // a whole block's lanes, or none
            break;
        const Piece8 p(a, row0, i0 + u * kBlock);
        unsigned top = top_of(x[u]);
        const bool special = __any(top >= kInfBits);   // NaN or an infinity in the wave
        if (special) {
            top = 0;
#pragma unroll
            for (int k = 0; k < kOct; ++k) {
                const unsigned b = __float_as_uint(x[u].at(k)) & 0x7fffffffu;
                top = max(top, b < kInfBits ? b : 0);
            }
        }
        const unsigned byte = scale_byte(block_max(top));
        const float s = scale_of(byte);
        unsigned w[2] = {codes_of(x[u], 0, s), codes_of(x[u], 1, s)};
        if (special) {
#pragma unroll
            for (int k = 0; k < kOct; ++k)
                if ((__float_as_uint(x[u].at(k)) & 0x7fffffffu) >= kInfBits)
                    w[k / 4] = (w[k / 4] & ~(0xffu << (8 * (k % 4)))) | 0x7fu << (8 * (k % 4));
        }
        uint8_t *q = a.codes + p.r * a.cols + p.c;
        if (p.n >= kOct)
            __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2_at1 *>(q));
        else
#pragma unroll
            for (int k = 0; k < kOct; ++k)
                if (k < p.n)
                    q[k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
        if (p.lane % kLanes == 0)
            a.scales[p.r * a.blocks + p.lane / kLanes] = (uint8_t)byte;
    }
}

// Eight codes' values in memory.
__device__ __forceinline__ void put_values(uint16_t *p, int n, u32x2 w, float s)
{
    unsigned v[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        v[2 * k] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[k], s, false));
        v[2 * k + 1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[k], s, true));
    }
    if (n >= kOct) {
        __builtin_nontemporal_store(u32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<u32x4_at2 *>(p));
        return;
    }
#pragma unroll
    for (int k = 0; k < kOct; ++k)
        if (k < n)
            p[k] = (uint16_t)(v[k / 2] >> (16 * (k % 2)));
}
__device__ __forceinline__ void put_values(float *p, int n, u32x2 w, float s)
{
    float x[kOct];
    widen_codes(w.x, s, x);
    widen_codes(w.y, s, x + 4);
    if (n >= kOct) {
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4_at4 *>(p));
        __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4_at4 *>(p + 4));
        return;
    }
    store_n(p, n, x);
}

template <typename T>
__global__ __launch_bounds__(kBlock) void unpack_kernel(Act8Args a, int64_t row0, uint32_t total)
{
    const uint32_t i0 = blockIdx.x * (kBlock * kTurns) + threadIdx.x;
    u32x2 w[kTurns];
    unsigned byte[kTurns];
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        const Piece8 p(a, row0, min(i0 + u * kBlock, total - 1));
        const uint8_t *q = a.codes + p.r * a.cols + p.c;
        byte[u] = a.scales[p.r * a.blocks + p.lane / kLanes];
        w[u] = u32x2{0, 0};
        if (p.n >= kOct)
            w[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_at1 *>(q));
        else
#pragma unroll
            for (int k = 0; k < kOct; ++k)
                if (k < p.n)
                    w[u][k / 4] |= (unsigned)q[k] << (8 * (k % 4));
    }
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        if (i0 + u * kBlock >= total)
            break;
        const Piece8 p(a, row0, i0 + u * kBlock);
        put_values(static_cast<T *>(a.x) + p.r * a.stride + p.c, p.n, w[u], scale_of(byte[u]));
    }
}

// f(first row, lanes) for launches whose threads 32 bits count.
template <typename F>
void each_launch(const Act8Args &a, F f)
{
    const int64_t lanes = (int64_t)a.blocks * kLanes, most = (int64_t(1) << 31) / lanes;
    for (int64_t r = 0; r < a.rows; r += most) {
        const uint32_t total = (uint32_t)(std::min(most, a.rows - r) * lanes);
        f(dim3((total + kBlock * kTurns - 1) / (kBlock * kTurns)), r, total);
    }
}

}  // namespace

int launch_act8_pack(const Act8Args &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    each_launch(a, [&](dim3 grid, int64_t r, uint32_t total) {
        if (a.dtype == ZERO_F32)
            hipLaunchKernelGGL((pack_kernel<float>), grid, dim3(kBlock), 0, st, a, r, total);
        else
            hipLaunchKernelGGL((pack_kernel<uint16_t>), grid, dim3(kBlock), 0, st, a, r, total);
    });
    return hipGetLastError();
}

int launch_act8_unpack(const Act8Args &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    each_launch(a, [&](dim3 grid, int64_t r, uint32_t total) {
        if (a.dtype == ZERO_F32)
            hipLaunchKernelGGL((unpack_kernel<float>), grid, dim3(kBlock), 0, st, a, r, total);
        else
            hipLaunchKernelGGL((unpack_kernel<uint16_t>), grid, dim3(kBlock), 0, st, a, r, total);
    });
    return hipGetLastError();
}

}  // namespace zero
