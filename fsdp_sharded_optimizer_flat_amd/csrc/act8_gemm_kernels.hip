// act8_gemm_kernels.hip -- a weight's gradient from an 8-bit activation checkpoint:
// d_w[o][c] = sum_r d_y[r][o] x'[r][c] on the matrix cores.
//
// Both factors lie in memory by rows r, the index summed over, so a lane of a
// matrix instruction needs eight of one column: tiles go to LDS as they lie (codes
// widened to bf16 on the way, one instruction for two codes and their scale, exact)
// and come back transposed (ds_read_b64_tr_b16: 16 lanes read four rows of 16
// columns, each gets a column).  Rows of a tile are cut into pairs of 16-byte
// chunks, pair p of row r at place p ^ (r & 7), so that the rows that one read
// touches lie in different banks.  Which of a step's 32 rows a lane holds is the
// same for both factors and otherwise free: lanes 16 g .. 16 g + 15 hold rows 4 g ..
// 4 g + 3 and 16 more.
#include <algorithm>

#include "act8_device.h"

namespace zero {
namespace {

using namespace dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kRows = 64;   // rows r of a tile

__device__ __forceinline__ unsigned widen_pair(unsigned w, float s, bool high)
{
    return __builtin_bit_cast(unsigned, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
}

// 16 bytes at p, of which n are within the array.
__device__ __forceinline__ u32x4 load_within(const uint8_t *p, int64_t n)
{
    if (n >= 16)
        return *reinterpret_cast<const u32x4_at1 *>(p);
    unsigned w[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n)
            w[i / 4] |= (unsigned)p[i] << (8 * (i % 4));
    return u32x4{w[0], w[1], w[2], w[3]};
}

// A workgroup of four waves per B x B tile of d_w, a wave per quarter.  FAST: rows
// of both factors are whole 16-byte chunks at 16-byte addresses.
template <int B, bool FAST, typename O>
__global__ __launch_bounds__(256, 1) void weight_grad_kernel(Act8GradArgs a)
{
    constexpr int N = B / 32;                    // 16 x 16 products of a wave, by rows and by columns
    constexpr int RowBytes = B * 2, Pairs = B / 16;
    constexpr int XPer = kRows * Pairs / 256, YPer = 2 * XPer;
    constexpr int Bytes = kRows * RowBytes;
    __shared__ __attribute__((aligned(16))) char sh[4 * Bytes];   // x', d_y; two tiles each
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int c0 = blockIdx.x * B, o0 = blockIdx.y * B;
    const int tiles = (int)((a.rows + kRows - 1) / kRows);
    const int per = (tiles + a.splits - 1) / a.splits;
    const int first = blockIdx.z * per, n = min(per, tiles - first);

    // A tile on its way: chunk i of x' and of d_y in registers.  Rows behind the last
    // are zeros; columns past a row's end may hold the next row's, which reach no
    // output.
    u32x4 xr[XPer], yr[YPer];
    unsigned sr[XPer];
    struct Source {
        const uint8_t *x, *s, *y;
        int64_t left;                        // rows from the tile's first on; <= 0: none
        __amdgpu_buffer_rsrc_t xw, sw, yw;   // FAST: bounded to the arrays
    };
    auto source = [&](int t) {
        Source f;
        const int64_t r0 = (int64_t)(first + t) * kRows;
        f.left = a.rows - r0;
        f.x = a.codes + r0 * a.cols + c0;
        f.s = a.scales + r0 * a.blocks + c0 / kActBlock;
        f.y = reinterpret_cast<const uint8_t *>(a.d_y + r0 * a.dy_stride + o0);
        if constexpr (FAST) {
            auto window = [&](const uint8_t *p, int64_t bytes) {
                const int64_t n = f.left > 0 ? min(max(bytes, int64_t(0)), int64_t(0x7fffffff)) : 0;
                return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, (int)n, kRawBufferWord3);
            };
            f.xw = window(f.x, f.left * a.cols - c0);
            f.sw = window(f.s, f.left * a.blocks - c0 / kActBlock);
            f.yw = window(f.y, ((f.left - 1) * a.dy_stride + a.out - o0) * 2);
        }
        return f;
    };
    // Chunk i of a thread: XRows i (YRows i) rows below its first.
    constexpr int XRows = 256 / Pairs, YRows = 128 / Pairs;
    const int xrow = tid / Pairs, xpair = tid % Pairs, yrow = tid / (2 * Pairs), yoct = tid % (2 * Pairs);
    const int xoff = xrow * a.cols + xpair * 16, soff = xrow * a.blocks + xpair / 2;
    const int yoff = (yrow * (int)a.dy_stride + yoct * 8) * 2;   // used where FAST, which bounds the stride
    auto load_x = [&](const Source &f, int i) {
        if constexpr (FAST) {
            xr[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(f.xw, xoff, i * XRows * a.cols, 0));
            sr[i] = __builtin_amdgcn_raw_buffer_load_b8(f.sw, soff, i * XRows * a.blocks, 0);
        } else {
            const int r = xrow + i * XRows;
            const int64_t at = (int64_t)r * a.cols + xpair * 16, sat = (int64_t)r * a.blocks + xpair / 2;
            xr[i] = load_within(f.x + at, r < f.left ? f.left * a.cols - c0 - at : 0);
            sr[i] = r < f.left && sat < f.left * a.blocks - c0 / kActBlock ? f.s[sat] : 0;
        }
    };
    auto load_y = [&](const Source &f, int i) {
        if constexpr (FAST) {
            yr[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  f.yw, yoff, i * YRows * (int)a.dy_stride * 2, 0));
        } else {
            const int r = yrow + i * YRows;
            const int64_t at = (r * a.dy_stride + yoct * 8) * 2;
            yr[i] = load_within(f.y + at, r < f.left ? ((f.left - 1) * a.dy_stride + a.out - o0) * 2 - at : 0);
        }
    };
    // Where a thread's first chunks go in a tile (the rows below are multiples of 8
    // further, so their places differ by whole rows), where a lane reads: its row of the
    // first four and product 0's columns, product t's being this ^ 32 t.  All change to
    // the other tile by ^ Bytes.
    static_assert(XRows % 8 == 0 && YRows % 8 == 0, "");
    int xto = xrow * RowBytes + ((xpair ^ (xrow & 7)) * 32);
    int yto = 2 * Bytes + yrow * RowBytes + ((yoct / 2 ^ (yrow & 7)) * 32) + yoct % 2 * 16;
    const int row = lane / 16 * 4 + lane % 16 / 4;
    int xat = row * RowBytes + ((wave % 2 * N ^ (row & 7)) * 32) + lane % 4 * 8;
    int yat = 2 * Bytes + row * RowBytes + ((wave / 2 * N ^ (row & 7)) * 32) + lane % 4 * 8;
    auto store_x = [&](int i) {
        const float s = __uint_as_float(sr[i] << 23);
        const unsigned w[4] = {xr[i].x, xr[i].y, xr[i].z, xr[i].w};
        unsigned v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = widen_pair(w[j / 2], s, j % 2);
        u32x4 *q = reinterpret_cast<u32x4 *>(sh + xto + i * XRows * RowBytes);
        q[0] = u32x4{v[0], v[1], v[2], v[3]};
        q[1] = u32x4{v[4], v[5], v[6], v[7]};
    };
    auto store_y = [&](int i) { *reinterpret_cast<u32x4 *>(sh + yto + i * YRows * RowBytes) = yr[i]; };
    auto column = [&](int at, int t, int half) {
        typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
        union {
            i16x4 h[2];
            bf16x8 v;
        } u;
        lds_char *p = (lds_char *)sh + (at ^ t * 32);
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p + half * 32 * RowBytes));
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p + (half * 32 + 16) * RowBytes));
        return u.v;
    };
    // A tile's products in 2 N groups: group g = half N + i multiplies columns i of
    // that half's rows with all of d_y's.  x' is read kAhead groups before, a half's d_y
    // during the half before.
    constexpr int kGroups = 2 * N, kAhead = 3;
    bf16x8 x[4], y[2][N];
    f32x4 acc[N][N] = {};   // [columns][out]
    if (n > 0) {
        for (int t = 0; t < 2; ++t) {
            const Source f = source(t);
#pragma unroll
            for (int i = 0; i < XPer; ++i)
                load_x(f, i);
#pragma unroll
            for (int i = 0; i < YPer; ++i)
                load_y(f, i);
            if (t == 1)
                break;
#pragma unroll
            for (int i = 0; i < XPer; ++i)
                store_x(i);
#pragma unroll
            for (int i = 0; i < YPer; ++i)
                store_y(i);
        }
        xto ^= Bytes, yto ^= Bytes;
        __syncthreads();
#pragma unroll
        for (int g = 0; g < kAhead; ++g)
            x[g] = column(xat, g, 0);
#pragma unroll
        for (int j = 0; j < N; ++j)
            y[0][j] = column(yat, j, 0);
        for (int t = 0; t < n; ++t) {
            const Source f = source(t + 2);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                if (g == kGroups - kAhead) {
                    __syncthreads();   // the next tile is there, this one is read
                    xat ^= Bytes, yat ^= Bytes, xto ^= Bytes, yto ^= Bytes;
                }
                __builtin_amdgcn_sched_barrier(0);
                const int ahead = (g + kAhead) % kGroups;
                x[ahead % 4] = column(xat, ahead % N, ahead / N);
                if (g < N)
                    y[1][g] = column(yat, g, 1);
                else
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (j * kAhead / N == g - (kGroups - kAhead))
                            y[0][j] = column(yat, j, 0);
                // the next tile's chunks to LDS, the one's after it on their way
                if (g < YPer) {
                    store_y(g);
                    load_y(f, g);
                }
                if (g % 3 == 1 && g / 3 < XPer) {
                    store_x(g / 3);
                    load_x(f, g / 3);
                }
#pragma unroll
                for (int j = 0; j < N; ++j)
                    acc[g % N][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[g % 4], y[g / N][j], acc[g % N][j], 0, 0, 0);
            }
        }
    }
    // a lane holds four neighbouring columns of a row of d_w
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = c0 + wave % 2 * (B / 2) + i * 16 + lane / 16 * 4;
            const int o = o0 + wave / 2 * (B / 2) + j * 16 + lane % 16;
            if (o >= a.out || c >= a.cols)
                continue;
            const int m = min(a.cols - c, 4);
            float v[4] = {acc[i][j].x, acc[i][j].y, acc[i][j].z, acc[i][j].w};
            if (a.splits > 1) {
                float *p = a.parts + ((int64_t)blockIdx.z * a.out + o) * a.columns + c;
                *reinterpret_cast<f32x4 *>(p) = acc[i][j];
                continue;
            }
            put4(static_cast<O *>(a.d_w) + (int64_t)o * a.w_stride + c, m, v, a.accumulate);
        }
}

// The parts of each element added in order; four columns to a thread.
template <typename O>
__global__ __launch_bounds__(kBlock) void join_splits_kernel(Act8GradArgs a)
{
    const int quads = a.columns / 4;
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (i >= (int64_t)quads * a.out)
        return;
    const int o = (int)(i / quads), c = (int)(i - (int64_t)o * quads) * 4;
    f32x4 sum = {};
    for (int s = 0; s < a.splits; ++s)
        sum += *reinterpret_cast<const f32x4 *>(a.parts + ((int64_t)s * a.out + o) * a.columns + c);
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
    put4(static_cast<O *>(a.d_w) + (int64_t)o * a.w_stride + c, min(a.cols - c, 4), v, a.accumulate);
}

template <int B, typename O>
void weight_grad_of(const Act8GradArgs &a, hipStream_t st)
{
    const dim3 grid((a.cols + B - 1) / B, (a.out + B - 1) / B, a.splits);
    const bool fast = a.out % 8 == 0 && a.dy_stride % 8 == 0 && a.dy_stride < 1 << 23 && a.cols % 16 == 0 &&
                      (reinterpret_cast<uintptr_t>(a.d_y) | reinterpret_cast<uintptr_t>(a.codes)) % 16 == 0;
    if (fast)
        hipLaunchKernelGGL((weight_grad_kernel<B, true, O>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((weight_grad_kernel<B, false, O>), grid, dim3(256), 0, st, a);
    if (a.splits > 1)
        hipLaunchKernelGGL((join_splits_kernel<O>), dim3((unsigned)(((int64_t)a.columns / 4 * a.out + kBlock - 1) / kBlock)),
                           dim3(kBlock), 0, st, a);
}

}  // namespace

Act8Split act8_split(int64_t rows, int64_t out, int64_t cols)
{
    auto tiles = [&](int64_t b) { return ((out + b - 1) / b) * ((cols + b - 1) / b); };
    if (tiles(256) >= 160)
        return {256, 1};
    const int64_t steps = (rows + kRows - 1) / kRows;
    const int64_t want = (512 + tiles(128) - 1) / tiles(128);
    const int64_t s = std::max<int64_t>(1, std::min(want, steps / 4));
    return {128, (int32_t)s};
}

int launch_act8_weight_grad(const Act8GradArgs &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    by_types(ZERO_F32, a.w_dtype, [&](auto, auto o) {
        if (a.tile == 256)
            weight_grad_of<256, decltype(o)>(a, st);
        else
            weight_grad_of<128, decltype(o)>(a, st);
    });
    return hipGetLastError();
}

}  // namespace zero
