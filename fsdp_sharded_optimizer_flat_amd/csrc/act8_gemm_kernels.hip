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
//
// Bound by the matrix cores' feeding: 8192 x 14336 x 4096 into bf16 takes 774 to 860 us,
// 1.12 to 1.24 PFLOP/s, as the clock goes, where the library's product of two bf16 matrices takes 950 to
// 1040; 8192 x 4096 x 4096 225 (230), with products under way in 51 % of the cycles and
// LDS busy in 32 %.  Small outputs have too few tiles for the device and are bound by a
// tile's latency: 1023 x 1280 x 1280 takes 15.7 us on 100 compute units (library: 20).
#include <algorithm>

#include "act8_device.h"

namespace zero {
namespace {

using namespace dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kRows = 64;   // rows r of a tile

__device__ __forceinline__ unsigned widen_pair(unsigned w, float s, bool high)
{
    return __builtin_bit_cast(unsigned, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
}

// v's bytes moved down by n > 0, zeros (16 and more: only zeros) behind them.
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int n)
{
    const int bits = min(n, 16) * 8;
    const uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
    const uint64_t l = bits < 64 ? lo >> bits | hi << 1 << (63 - bits) : bits < 128 ? hi >> (bits - 64) : 0;
    const uint64_t h = bits < 64 ? hi >> bits : 0;
    return u32x4{(unsigned)l, (unsigned)(l >> 32), (unsigned)h, (unsigned)(h >> 32)};
}

// The tile and share of the rows that a workgroup takes, and its part (none: -1).
// Workgroups go to the eight dies in turn; each die takes neighbours among the tiles, so
// that a factor's tiles stay in the L2 of few dies.
constexpr unsigned kDies = 8;
__device__ __forceinline__ void place_of(const Act8GradArgs &a, int tile, int &ct, int &ot, int &split, int &part)
{
    const unsigned whole = (unsigned)a.whole;
    const bool shared = blockIdx.x >= whole;
    const unsigned b = shared ? blockIdx.x - whole : blockIdx.x, all = shared ? gridDim.x - whole : whole;
    const unsigned die = b % kDies, q = all / kDies, r = all % kDies;
    unsigned i = die * q + min(die, r) + b / kDies;
    const unsigned cts = (unsigned)(a.cols + tile - 1) / tile;
    split = 0, part = -1;
    if (shared) {
        const unsigned tiles = all / (unsigned)a.splits;
        part = (int)i;
        split = (int)(i / tiles);
        i = whole + i % tiles;
    }
    ct = (int)(i % cts);
    ot = (int)(i / cts);
}

// A workgroup of four waves per B x B tile of d_w, a wave per quarter.  FAST: rows
// of both factors are whole 16-byte chunks at 16-byte addresses, read through buffer
// descriptors, whose bounds replace the general path's (8192 x 14336 x 4096 with whole
// tiles: 825 us, by the general path 866).
template <int B, bool FAST, typename O>
__global__ __launch_bounds__(256, 1) void weight_grad_kernel(Act8GradArgs a)
{
    constexpr int N = B / 32;                    // 16 x 16 products of a wave, by rows and by columns
    constexpr int RowBytes = B * 2, Pairs = B / 16;
    constexpr int XPer = kRows * Pairs / 256, YPer = 2 * XPer;
    constexpr int Bytes = kRows * RowBytes;
    // Tiles on their way in registers: a small tile's products are over before memory
    // answers (8192 x 1280 x 1280, 100 workgroups: 128 us with one, 83 with three).
    constexpr int kDepth = B == 256 ? 1 : 3;
    __shared__ __attribute__((aligned(16))) char sh[4 * Bytes];   // x', d_y; two tiles each
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    int ct, ot, split, part;
    place_of(a, B, ct, ot, split, part);
    const int c0 = ct * B, o0 = ot * B;
    const int tiles = (int)((a.rows + kRows - 1) / kRows);
    const int per = part < 0 ? tiles : (tiles + a.splits - 1) / a.splits;
    const int first = split * per, n = min(per, tiles - first);

    // A tile on its way: chunk i of x' and of d_y in registers.  Rows behind the last
    // are zeros; columns past a row's end may hold the next row's, which reach no
    // output.  FAST: windows that end where the arrays do (what lies past them reads as
    // zero, also where the scalar offset alone is past it: tests/test_gpu_act8_windows.py
    // has NaN there).  Else a chunk that would reach past its array is read from the array's last
    // 16 bytes and shifted to its place before it is stored (settle).
    u32x4 xr[kDepth][XPer], yr[kDepth][YPer];
    unsigned sr[kDepth][XPer];
    struct Source {
        const uint8_t *x, *s, *y;            // from the tile's first row and column on
        int xend, send, yend;                // bytes from there to the arrays' ends, 2^31 - 1 at most
        __amdgpu_buffer_rsrc_t xw, sw, yw;
    };
    // The tile that is read next; behind the array's last, the last again, which is not
    // used (FAST: behind the workgroup's last, nothing).
    int ahead_of = first;
    const int64_t r0 = (int64_t)min(first, tiles - 1) * kRows, left = a.rows - r0;
    const uint8_t *xp = a.codes + r0 * a.cols + c0, *sp = a.scales + r0 * a.blocks + c0 / kActBlock;
    const uint8_t *yp = reinterpret_cast<const uint8_t *>(a.d_y + r0 * a.dy_stride + o0);
    int64_t xleft = left * a.cols - c0, sleft = left * a.blocks - c0 / kActBlock;
    int64_t yleft = ((left - 1) * a.dy_stride + a.out - o0) * 2;
    auto next_source = [&]() {
        // by scalar arithmetic of few steps: nothing else runs while it does
        auto bound = [](int64_t bytes) { return (uint64_t)bytes >> 31 ? 0x7fffffff : (int)bytes; };
        Source f;
        f.x = xp, f.s = sp, f.y = yp;
        f.xend = bound(xleft), f.send = bound(sleft), f.yend = bound(yleft);
        if constexpr (FAST) {
            if (ahead_of >= first + n)
                f.xend = f.send = f.yend = 0;
            auto window = [](const uint8_t *p, int n) {
                return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, n, kRawBufferWord3);
            };
            f.xw = window(f.x, f.xend), f.sw = window(f.s, f.send), f.yw = window(f.y, f.yend);
        }
        const int go = ++ahead_of < tiles ? kRows : 0;
        const int64_t dx = (int64_t)go * a.cols, ds = (int64_t)go * a.blocks, dy = (int64_t)go * (int)a.dy_stride * 2;
        xp += dx, sp += ds, yp += dy;
        xleft -= dx, sleft -= ds, yleft -= dy;
        return f;
    };
    // Chunk i of a thread: XRows i (YRows i) rows below its first.
    constexpr int XRows = 256 / Pairs, YRows = 128 / Pairs;
    const int xrow = tid / Pairs, xpair = tid % Pairs, yrow = tid / (2 * Pairs), yoct = tid % (2 * Pairs);
    const int xoff = xrow * a.cols + xpair * 16, soff = xrow * a.blocks + xpair / 2;
    const int yoff = (yrow * (int)a.dy_stride + yoct * 8) * 2;
    const int xstep = XRows * a.cols, sstep = XRows * a.blocks, ystep = YRows * (int)a.dy_stride * 2;
    auto load_x = [&](const Source &f, int d, int i) {
        if constexpr (FAST) {
            xr[d][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(f.xw, xoff, i * xstep, 0));
            sr[d][i] = __builtin_amdgcn_raw_buffer_load_b8(f.sw, soff, i * sstep, 0);
        } else {
            xr[d][i] = *reinterpret_cast<const u32x4_at1 *>(f.x + i * xstep + min(xoff, f.xend - 16 - i * xstep));
            sr[d][i] = (f.s + i * sstep)[min(soff, f.send - 1 - i * sstep)];
        }
    };
    auto load_y = [&](const Source &f, int d, int i) {
        if constexpr (FAST)
            yr[d][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(f.yw, yoff, i * ystep, 0));
        else
            yr[d][i] = *reinterpret_cast<const u32x4_at1 *>(f.y + i * ystep + min(yoff, f.yend - 16 - i * ystep));
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
    // Before a tile is stored, if it is one at the arrays' ends: chunks read early to
    // their places.
    auto settle = [&](const Source &f, int d) {
        if (f.xend >= (kRows - 1) * a.cols + B && f.yend >= ((kRows - 1) * (int)a.dy_stride + B) * 2)
            return;
#pragma unroll
        for (int i = 0; i < XPer; ++i) {
            const int over = xoff + i * xstep - (f.xend - 16);
            if (over > 0) {
                xr[d][i] = shift_down(xr[d][i], over);
                sr[d][i] = over >= 16 ? 0 : sr[d][i];   // no row: not even a NaN scale
            }
        }
#pragma unroll
        for (int i = 0; i < YPer; ++i) {
            const int over = yoff + i * ystep - (f.yend - 16);
            if (over > 0)
                yr[d][i] = shift_down(yr[d][i], over);
        }
    };
    // Words w0 .. w1 - 1 of chunk i's eight of values, to LDS by fours.
    unsigned wide[8];
    auto store_x = [&](int d, int i, int w0, int w1) {
        const float s = __uint_as_float(sr[d][i] << 23);
        const unsigned w[4] = {xr[d][i].x, xr[d][i].y, xr[d][i].z, xr[d][i].w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j >= w0 && j < w1)
                wide[j] = widen_pair(w[j / 2], s, j % 2);
        u32x4 *q = reinterpret_cast<u32x4 *>(sh + xto + i * XRows * RowBytes);
        if (w0 < 4 && w1 >= 4)
            q[0] = u32x4{wide[0], wide[1], wide[2], wide[3]};
        if (w1 == 8)
            q[1] = u32x4{wide[4], wide[5], wide[6], wide[7]};
    };
    auto store_y = [&](int d, int i) {
        *reinterpret_cast<u32x4 *>(sh + yto + i * YRows * RowBytes) = yr[d][i];
    };
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
        Source held[kDepth];   // of the chunks in registers
        auto fetch = [&](int d) {
            held[d] = next_source();
#pragma unroll
            for (int i = 0; i < XPer; ++i)
                load_x(held[d], d, i);
#pragma unroll
            for (int i = 0; i < YPer; ++i)
                load_y(held[d], d, i);
        };
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
            fetch(d);
        if constexpr (!FAST)
            settle(held[0], 0);
#pragma unroll
        for (int i = 0; i < XPer; ++i)
            store_x(0, i, 0, 8);
#pragma unroll
        for (int i = 0; i < YPer; ++i)
            store_y(0, i);
        fetch(0);
        xto ^= Bytes, yto ^= Bytes;
        __syncthreads();
#pragma unroll
        for (int g = 0; g < kAhead; ++g)
            x[g] = column(xat, g, 0);
#pragma unroll
        for (int j = 0; j < N; ++j)
            y[0][j] = column(yat, j, 0);
        auto step = [&](int d, int t) {   // tile t; d: where tile t + 1 is held
            if constexpr (!FAST)
                settle(held[d], d);
            const Source f = next_source();   // chunk by chunk in the places of held[d]'s
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                if (g == kGroups - kAhead) {
                    __syncthreads();   // the next tile is there, this one is read
                    xat ^= Bytes, yat ^= Bytes, xto ^= Bytes, yto ^= Bytes;
                }
                // work for the shadow of each product: two reads of x', of d_y, the next
                // tile's chunks to LDS, a later one's on their way
                auto beside = [&](int j) {
                    const int ahead = (g + kAhead) % kGroups;
                    if (j == 0)
                        x[ahead % 4] = column(xat, ahead % N, ahead / N);
                    if (g < N && j == 1)
                        y[1][g] = column(yat, g, 1);
                    if (g >= kGroups - kAhead && (j * kAhead + kAhead - 1) / N == g - (kGroups - kAhead))
                        y[0][j] = column(yat, j, 0);
                    if (g < YPer && j == N / 2) {
                        store_y(d, g);
                        load_y(f, d, g);
                    }
                    if (g % 3 == 1 && g / 3 < XPer) {
                        store_x(d, g / 3, j * 8 / N, (j + 1) * 8 / N);
                        if (j == N - 1)
                            load_x(f, d, g / 3);
                    }
                };
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
                    acc[g % N][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[g % 4], y[g / N][j], acc[g % N][j], 0, 0, 0);
                    beside(j);
                }
            }
            held[d] = f;
        };
        if constexpr (kDepth == 1) {
            for (int t = 0; t < n; ++t)
                step(0, t);
        } else {
            for (int t = 0; t < n; t += kDepth)
#pragma unroll
                for (int i = 0; i < kDepth; ++i)
                    if (t + i < n)
                        step((i + 1) % kDepth, t + i);
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
            if (part >= 0) {
                float *p = a.parts + (int64_t)part * (B * B) + (o - o0) * B + c - c0;
                *reinterpret_cast<f32x4 *>(p) = acc[i][j];
                continue;
            }
            put4(static_cast<O *>(a.d_w) + (int64_t)o * a.w_stride + c, m, v, a.accumulate);
        }
}

// Arrays of fewer than 16 bytes: an element to a thread.
template <typename O>
__global__ __launch_bounds__(kBlock) void weight_grad_of_few_kernel(Act8GradArgs a)
{
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (i >= (int64_t)a.out * a.cols)
        return;
    const int o = (int)(i / a.cols), c = (int)(i - (int64_t)o * a.cols);
    float sum[4] = {};
    for (int64_t r = 0; r < a.rows; ++r) {
        float x[4];
        widen_codes(a.codes[r * a.cols + c], scale_of(a.scales[r * a.blocks + c / kActBlock]), x);
        sum[0] += widen<uint16_t>(a.d_y[r * a.dy_stride + o]) * widen<uint16_t>(to_bf16(x[0]));
    }
    put4(static_cast<O *>(a.d_w) + (int64_t)o * a.w_stride + c, 1, sum, a.accumulate);
}

// The parts of each element of the shared tiles added in order; four columns to a
// thread, a workgroup per kBlock of them within a tile.
template <int B, typename O>
__global__ __launch_bounds__(kBlock) void join_splits_kernel(Act8GradArgs a)
{
    constexpr unsigned Groups = B * B / 4 / kBlock;   // of a tile
    const unsigned t = blockIdx.x / Groups, quad = blockIdx.x % Groups * kBlock + threadIdx.x;
    const unsigned tiles = gridDim.x / Groups, cts = (unsigned)(a.cols + B - 1) / B, tile = (unsigned)a.whole + t;
    const int o = (int)(tile / cts * B + quad / (B / 4)), c = (int)(tile % cts * B + quad % (B / 4) * 4);
    if (o >= a.out || c >= a.cols)
        return;
    f32x4 sum = {};
    for (int s = 0; s < a.splits; ++s)
        sum += *reinterpret_cast<const f32x4 *>(a.parts + ((int64_t)s * tiles + t) * (B * B) + quad * 4);
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
    put4(static_cast<O *>(a.d_w) + (int64_t)o * a.w_stride + c, min(a.cols - c, 4), v, a.accumulate);
}

template <int B, typename O>
void weight_grad_of(const Act8GradArgs &a, hipStream_t st)
{
    const unsigned shared = (unsigned)Act8Split{B, a.splits, a.whole}.shared(a.out, a.cols);
    const dim3 grid((unsigned)a.whole + shared * (unsigned)a.splits);
    const bool fast = a.out % 8 == 0 && a.dy_stride % 8 == 0 && a.cols % 16 == 0 &&
                      (reinterpret_cast<uintptr_t>(a.d_y) | reinterpret_cast<uintptr_t>(a.codes)) % 16 == 0;
    if (fast)
        hipLaunchKernelGGL((weight_grad_kernel<B, true, O>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((weight_grad_kernel<B, false, O>), grid, dim3(256), 0, st, a);
    if (shared > 0)
        hipLaunchKernelGGL((join_splits_kernel<B, O>), dim3(shared * (B * B / 4 / kBlock)), dim3(kBlock), 0, st, a);
}

}  // namespace

// Tiles of 256 x 256 read LDS half as often for a product as those of 128 x 128, but
// small outputs have few of them; rows are split over workgroups where there are few
// tiles of either kind, at the price of the parts' way through memory; or only those of
// the last tiles that do not fill the device (8192 x 14336 x 4096, 128 of 896: 850 us
// without, 815 with it; 8192 x 4095 x 4097, 16 of 272: 400 and 276; 36 random sizes where
// this is chosen, 0.99 to 1.42 times as fast, 1.2 in the middle).  The least of these
// estimates, in us, fitted to sweeps over tiles and splits (what they give | what was
// measured):
//      rows x out x cols      256 / 1     256 / split     128 / 1     128 / split
//   8192 x 4096 x  4096      223 | 225    272 | 255 (2)    282 | 279    332 | 326 (2)
//   4096 x 1280 x  5120      118 | 107     81 |  72 (2)     74 |  75     97 |  93 (2)
//   8192 x 1280 x  1280      223 | 194     56 |  50 (8)     83 |  83     50 |  48 (4)
//   2048 x 1280 x  1280       65 |  58     36 |  33 (8)     26 |  26     23 |  25 (2)
//   1024 x 1280 x  1280       38 |  35     29 |  30 (4)     16 |  16     18 |  20 (2)
//  16384 x   64 x    64      434 | 369     35 |  29 (32)   160 | 157     21 |  20 (24)
Act8Split act8_split(int64_t rows, int64_t out, int64_t cols)
{
    const int64_t steps = std::max<int64_t>(1, (rows + kRows - 1) / kRows);
    Act8Split best{128, 1, 0};
    double least = 1e300;
    for (int32_t tile : {256, 128}) {
        const int64_t tiles = ((out + tile - 1) / tile) * ((cols + tile - 1) / tile);
        // one large tile fits a compute unit, two small ones, which slow each other
        const int64_t round = tile == 256 ? 256 : 512;
        auto time = [&](int64_t groups, int64_t per) {
            return tile == 256    ? (double)((groups + 255) / 256) * (1.65 * (double)per + 12.0)
                   : groups <= 256 ? 0.6 * (double)per + 6.5
                                   : (double)((groups + 511) / 512) * (1.05 * (double)per + 6.5);
        };
        for (int64_t s = 1; s <= std::min<int64_t>(steps, 64); ++s) {
            const int64_t per = (steps + s - 1) / s;
            if ((steps + per - 1) / per != s)
                continue;   // the last workgroup would have none
            // all tiles shared, or those of the last round
            for (int64_t whole : {s == 1 ? tiles : 0, tiles / round * round}) {
                const int64_t rest = tiles - whole;
                if (rest > 0 && s == 1)
                    continue;
                double t = rest < tiles ? time(whole, steps) : 0.0;
                if (rest > 0)
                    t += time(rest * s, per) + 3.0 + 0.2 * (double)s +
                         1e-6 * (double)(s * std::min(rest * tile * tile, out * cols));
                if (t < least)
                    least = t, best = {tile, (int32_t)s, (int32_t)whole};
            }
        }
    }
    return best;
}

int launch_act8_weight_grad(const Act8GradArgs &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    by_types(ZERO_F32, a.w_dtype, [&](auto, auto o) {
        // (no rows: the tiled kernel writes zeros, of any size)
        if (a.rows > 0 && (a.rows * a.cols < 16 || (a.rows - 1) * a.dy_stride + a.out < 8))
            hipLaunchKernelGGL((weight_grad_of_few_kernel<decltype(o)>),
                               dim3((unsigned)(((int64_t)a.out * a.cols + kBlock - 1) / kBlock)), dim3(kBlock), 0, st, a);
        else if (a.tile == 256)
            weight_grad_of<256, decltype(o)>(a, st);
        else
            weight_grad_of<128, decltype(o)>(a, st);
    });
    return hipGetLastError();
}

}  // namespace zero
