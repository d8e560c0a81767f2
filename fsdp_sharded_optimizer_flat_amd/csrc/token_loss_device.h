// token_loss_device.h -- what the kernels of the token losses share: rows cut
// into 16-byte chunks, running sums of exponentials, rows mapped to gradients,
// rows held in registers.
//
// All work is done in binary logarithms: with c = scale * log2(e) a logit l
// counts as t = c l - R, R = fl(c m) for a reference logit m, and 2^t is one
// v_exp_f32.  One fused multiply-add forms t with a single rounding relative to
// the reference, so the error of 2^t grows with l's distance from the
// reference only.  A lane keeps the sum of 2^t over its elements in one pass:
// its reference is the largest logit of its first group, raised (the sum
// rescaled) only when a group exceeds it by more than kHeadroom binary orders
// -- sums stay far inside binary32's range, and after the first groups almost
// no group raises it.  R's own rounding cancels between the sums and what is
// read off them while it is small; for references with |c m| > 2^20 (rows of huge
// logits, or parts of rows masked with the type's lowest value, where c m could
// even leave binary32's range) t = (l - m) c is taken instead.
//
// Bound: HBM.  A forward pass reads each logit once, a backward pass reads and
// writes, a fused call too (it holds the row in registers).  A bf16 element is 2
// bytes against 7 to 10 vector issue slots (widen 1, max 1, fma 1, exp 2, add 1,
// bookkeeping 1; entropy: clamp, product and sum 1 each): with the entropy the
// vector units are as busy as the memory (counters: 0.92 of their cycles at 6.5
// TB/s), so no term may be added lightly.  A single row waits for its one compute
// unit instead (1 x 50304: 5 of 10.9 us).
// Log probabilities on one MI355X (a sweep that reads and writes reaches 6.4 to 6.7
// TB/s there): forward with entropy, 4096 x 128256 bf16, 162 us, 6.5 TB/s;
// backward with entropy, 2048 x 50304 fp32, 124 us, 6.6 TB/s, 2048 x 128256 bf16,
// 165 us, 6.4 TB/s; loss and gradient, 8192 x 128256 bf16, 746 us, 5.6 TB/s.
#pragma once

#include <algorithm>

#include "device_common.h"
#include "token_loss.h"

namespace zero {
namespace dev {

constexpr int kNT = kLossBlock;
constexpr int kNW = kNT / kWave;
constexpr float kInf = __builtin_inff();
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLowest = -3.40282346638528859812e38f;
constexpr float kHeadroom = 10.0f;      // binary orders a group may exceed a lane's reference
constexpr float kBig = 0x1p20f;         // |c m| beyond it: t = (l - m) c
constexpr float kTiny = -1000.0f;       // t of a probability that is zero, for products with it

// -- loading -------------------------------------------------------------------------

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr int kLine = 128;   // bytes of a cache line

// 16 bytes of a row: W elements.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    static constexpr int W = 8;
    u32x4 r;
    __device__ __forceinline__ void clear() { r = u32x4{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u}; }   // -inf
    __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const u32x4 *>(p); }
    __device__ __forceinline__ void stream(const uint16_t *p)
    {
        r = ld_stream(reinterpret_cast<const u32x4 *>(p));
    }
    __device__ __forceinline__ void widen(float (&x)[W]) const
    {
        // as a conversion: the compiler then knows that no value is a signalling
        // NaN and takes their maximum without quieting each first
        const f32x8 v = __builtin_convertvector(__builtin_bit_cast(bf16x8, r), f32x8);
#pragma unroll
        for (int i = 0; i < W; ++i)
            x[i] = v[i];
    }
};
template <>
struct Chunk<float> {
    static constexpr int W = 4;
    f32x4 r;
    __device__ __forceinline__ void clear() { r = f32x4{-kInf, -kInf, -kInf, -kInf}; }
    __device__ __forceinline__ void load(const float *p) { r = *reinterpret_cast<const f32x4 *>(p); }
    __device__ __forceinline__ void stream(const float *p)
    {
        r = ld_stream(reinterpret_cast<const f32x4 *>(p));
    }
    __device__ __forceinline__ void widen(float (&x)[W]) const
    {
        x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
    }
};

// A chunk's gradients, each rounded once.
template <typename T, int W>
__device__ __forceinline__ u32x4 pack_chunk(const float (&g)[W])
{
    if constexpr (sizeof(T) == 2)
        return u32x4{pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]),
                     pack_bf16x2(g[6], g[7])};
    else
        return u32x4{__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]),
                     __float_as_uint(g[3])};
}
// Stores 16 bytes at any element's address (gfx950 takes such stores), for
// gradients whose rows sit at another 16-byte phase than their logits: reading
// the logits unaligned instead measured slower (log probabilities, loss and gradient
// of 777 x 50257 fp32 in rows of 50304, the gradient's rows back to back: 70 us, and 80
// to 93 us with unaligned loads).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <typename T>
__device__ __forceinline__ void store_any(u32x4 v, T *p)
{
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any *>(p));
}
__device__ __forceinline__ void store_one(uint16_t *p, float g) { *p = to_bf16(g); }
__device__ __forceinline__ void store_one(float *p, float g) { *p = g; }

// A value at an address that is the same in every lane, read into a scalar
// register: only for arrays that the call does not write (its checks keep outputs
// apart from them).  Such a load does not queue behind the vector loads and stores.
template <typename T>
__device__ __forceinline__ T ld_uniform(const T *p)
{
    return *(const __attribute__((address_space(4))) T *)p;
}

// p, which is the same in every lane, in scalar registers.
template <typename T>
__device__ __forceinline__ T *scalar(const T *p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint64_t u = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
    return reinterpret_cast<T *>(u);
}
// `chunks` chunks from p on as a buffer: what lies past them is neither read nor
// written.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const T *p, int chunks)
{
    return __builtin_amdgcn_make_buffer_rsrc(scalar(p), 0, __builtin_amdgcn_readfirstlane(chunks) * 16,
                                             kRawBufferWord3);
}
// Stores chunk `tid` - skip of a window of `chunks` chunks from p on, nontemporal (the
// threads below skip store nothing: their offset wraps past the window).  Not written
// through to memory (sc1) as well: where waves share a cache line its halves then go
// out one by one (log probabilities, loss and gradient of 4096 x 128256 bf16, whole
// lines, 380 us so and 374 without; with waves that began anywhere in a line, 4096 x
// 128255, 457 and 422).  Without the nontemporal hint outputs beyond the memory-side
// cache lose (4096 x 128256: 413).  Each store has a window of its own, no offset in a scalar register:
// MI355X has stored what the next instruction wrote to the data registers of a
// 16-byte buffer store with such an offset (the compiler leaves no wait between the
// two then).
constexpr int kLossStorePolicy = 2;   // nt
template <typename T>
__device__ __forceinline__ void store_chunks(u32x4 v, T *p, int chunks, int skip = 0)
{
    __builtin_amdgcn_raw_buffer_store_b128(v, window(p, chunks), ((int)threadIdx.x - skip) * 16, 0,
                                           kLossStorePolicy);
}

// A row cut into 16-byte chunks, counted from the cache line (128 bytes) it starts
// in, so that waves that take 64 chunks of a row at a time read and write whole
// lines: chunk k holds elements k W - phase .. + W - 1, whole for full_lo <= k <
// full_hi; the one before and the one after may hold a few elements of the row and
// are read element by element.  (Counted from the 16 bytes it starts in: log
// probabilities, loss and gradient of 4096 x 128255 bf16 422 us, and 378 so; 777 x
// 50257 fp32, logits and gradient back to back, 70 and 64.)
template <typename T>
struct Row {
    static constexpr int W = Chunk<T>::W;
    const T *p;
    int vocab, phase, chunks, full_lo, full_hi;
    __device__ __forceinline__ Row() : p(nullptr), vocab(0), phase(0), chunks(0), full_lo(0), full_hi(0) {}
    __device__ __forceinline__ Row(const T *p_, int vocab_) : p(p_), vocab(vocab_)
    {
        phase = (int)((reinterpret_cast<uintptr_t>(p) & (kLine - 1)) / sizeof(T));
        chunks = (vocab + phase + W - 1) / W;
        full_lo = (phase + W - 1) / W;
        full_hi = max(full_lo, (vocab + phase) / W);
    }
    __device__ __forceinline__ const T *chunk(int k) const { return p + ((int64_t)k * W - phase); }
    __device__ __forceinline__ float at(int e) const { return grad_at<T>(p, e); }
    // Element of edge slot s (0 .. 2W-1: the head's, then the tail's) among
    // chunks [k0, k1), or -1.
    __device__ __forceinline__ int edge(int s, int k0, int k1) const
    {
        const int k = s < W ? full_lo - 1 : full_hi;
        const int e = k * W - phase + (s & (W - 1));
        const bool partial = s < W ? (phase & (W - 1)) != 0 : full_hi < chunks;
        return partial && k >= k0 && k < k1 && e >= 0 && e < vocab ? e : -1;
    }
};

// Chunks [lo, hi) of a row as a workgroup goes through them, NT threads at a time:
// its place c is chunk from + c, from being the line that lo lies in, so that the
// first `skip` places hold nothing (log probabilities of 4096 x 128255 bf16: 180 us
// where the first thread takes chunk lo, 167 so).
template <typename T>
struct Sweep {
    int lo, hi, skip, from, n;   // n: places
    __amdgpu_buffer_rsrc_t in;
    __device__ __forceinline__ Sweep(const Row<T> &row, int k0, int k1)
        : lo(max(k0, row.full_lo)), hi(max(min(k1, row.full_hi), lo)), skip(lo & (kLine / 16 - 1)), from(lo - skip),
          n(hi > lo ? hi - from : 0), in(window(row.chunk(lo), hi - lo))
    {
    }
    // Reads place first + tid, first being the same in every lane and 0 or at least
    // 64; what lies outside is not read (offsets below the first chunk wrap past
    // the window).
    __device__ __forceinline__ Chunk<T> read(int first) const
    {
        int at = ((int)threadIdx.x - skip) * 16 + (first ? kWave * 16 : 0);
        asm volatile("" : "+v"(at));   // in a register: the wrapped sum
        Chunk<T> ch;
        ch.r = __builtin_bit_cast(decltype(ch.r),
                                  __builtin_amdgcn_raw_buffer_load_b128(
                                      in, at, first ? (first - kWave) * 16 : 0, kLoadStreamPolicy));
        return ch;
    }
    // Makes a place outside -inf.
    __device__ __forceinline__ void trim(Chunk<T> &ch, int first, int threads) const
    {
        if (first == 0 || first + threads > n) {
            const int c = first + (int)threadIdx.x;
            if (c < skip || c >= n)
                ch.clear();
        }
    }
};

// -- running sums ------------------------------------------------------------------------

struct Scale {
    float c, gap, big;   // logits that span kHeadroom binary orders, and |m| beyond which |c m| > kBig
    __device__ __forceinline__ explicit Scale(float c_) : c(c_), gap(kHeadroom / c_), big(kBig / c_) {}
};

// t of logit l against reference m (r = fl(c m)).
__device__ __forceinline__ float rel(float l, float m, float r, const Scale &k)
{
    return __builtin_fabsf(m) > k.big ? (l - m) * k.c : __builtin_fmaf(l, k.c, -r);
}
// c m - fl(c m): what the sums' reference R is off the exact one by.
__device__ __forceinline__ float residue(float m, const Scale &k)
{
    return __builtin_fabsf(m) > k.big ? 0.0f : __builtin_fmaf(m, k.c, -(m * k.c));
}
// t of reference m against reference n, as the sums were formed: R of either is
// fl(c m), or c m itself beyond kBig.  Where one of them is of each kind (|c m|
// around 2^20, fl(c m) off by up to 2^-5 there) the difference of the two kinds counts.
__device__ __forceinline__ float shift_of(float m, float n, const Scale &k)
{
    return __builtin_fabsf(m) > k.big || __builtin_fabsf(n) > k.big ? (m - n) * k.c - residue(m, k) + residue(n, k)
                                                                    : m * k.c - n * k.c;
}
__device__ __forceinline__ float pow2(float t) { return __builtin_amdgcn_exp2f(t); }

struct Sum {
    float top;       // the largest logit seen
    float m, r;      // the reference and fl(c m)
    float thr;       // groups whose largest logit is above it raise the reference
    float s, a;      // sums of 2^t and of t 2^t
    bool big;        // of the wave: some lane's |c m| is beyond kBig
    __device__ __forceinline__ Sum() : top(-kInf), m(0), r(0), thr(-kInf), s(0), a(0), big(false) {}

    __device__ __forceinline__ void rebase(float n, const Scale &k)
    {
        if (s != 0.0f) {   // else nothing is added yet, and n may lie below m
            const float d = shift_of(m, n, k), f = pow2(d);
            a = f * (a + __builtin_fmaxf(d, kTiny) * s);
            s = s * f;
        }
        m = n;
        r = n * k.c;
    }

    // Adds N elements (every lane of the wave that is to add any calls it).  A
    // NaN among them makes the sum NaN (max ignores it).
    template <int N, bool ENT>
    __device__ __forceinline__ void add(const float (&x)[N], const Scale &k)
    {
        float g = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i)
            g = __builtin_fmaxf(g, x[i]);
        add_with_max<N, ENT>(x, g, k);
    }
    template <int N, bool ENT>
    __device__ __forceinline__ void add_with_max(const float (&x)[N], float g, const Scale &k)
    {
        top = __builtin_fmaxf(top, g);
        if (__any(g > thr)) {
            if (g > thr) {
                rebase(g, k);
                thr = g + k.gap;
            }
            big = __any(__builtin_fabsf(m) > k.big);
        }
        if (big)
            add_terms<N, ENT, true>(x, k);
        else
            add_terms<N, ENT, false>(x, k);
    }
    template <int N, bool ENT, bool BIG>
    __device__ __forceinline__ void add_terms(const float (&x)[N], const Scale &k)
    {
        // a group's sums apart from the lane's, as trees: they round less, and no
        // addition waits for the exponential before it
        float e[N], b[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = BIG ? rel(x[i], m, r, k) : __builtin_fmaf(x[i], k.c, -r);
            e[i] = pow2(t);
            if constexpr (ENT) {
                const float u = __builtin_fmaxf(t, kTiny);
                b[i] = 0.0f;
                if (i & 1)
                    b[i - 1] = __builtin_fmaf(e[i], u, b[i - 1]);
                else
                    b[i] = e[i] * u;
            }
        }
#pragma unroll
        for (int w = 1; w < N; w *= 2)
#pragma unroll
            for (int i = 0; i + w < N; i += 2 * w) {
                e[i] += e[i + w];
                if constexpr (ENT)
                    if (w > 1)
                        b[i] += b[i + w];
            }
        s += e[0];
        if constexpr (ENT)
            a += b[0];
    }
};

// The sum of a wave's or workgroup's lanes against the largest logit among
// them (kLowest at least), in a fixed order.
struct Total {
    float m, s, a;
    __device__ __forceinline__ bool empty() const { return s == 0.0f; }   // every logit -inf
};

// Over a wave, in every lane, in a fixed order: within rows of 16 lanes by
// exchanges between neighbours, then row by row to the last lane (data-parallel
// moves: a shuffle through LDS takes about ten times as long).
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float from_lane(float other, float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(other), __float_as_int(x), CTRL, ROWS,
                                                      0xf, false));
}
constexpr int kLaneXor1 = 0xb1, kLaneXor2 = 0x4e, kMirror8 = 0x141, kMirror16 = 0x140;
constexpr int kLastOfRow = 0x142, kLastOfHalf = 0x143;   // lane 15 / 31 to the next rows
template <typename F>
__device__ __forceinline__ float wave_reduce(float x, float neutral, F f)
{
    x = f(x, from_lane<kLaneXor1>(x, x));
    x = f(x, from_lane<kLaneXor2>(x, x));
    x = f(x, from_lane<kMirror8>(x, x));
    x = f(x, from_lane<kMirror16>(x, x));
    x = f(x, from_lane<kLastOfRow, 0xa>(neutral, x));
    x = f(x, from_lane<kLastOfHalf, 0xc>(neutral, x));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}
__device__ __forceinline__ float wave_max(float x)
{
    return wave_reduce(x, -kInf, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ float wave_add(float x)
{
    return wave_reduce(x, 0.0f, [](float a, float b) { return a + b; });
}

// One of several totals moved to reference m and added.
__device__ __forceinline__ void add_total(Total &t, const Total &o, const Scale &k)
{
    const float d = shift_of(o.m, t.m, k), f = pow2(d);
    t.a += f * (o.a + __builtin_fmaxf(d, kTiny) * o.s);
    t.s += f * o.s;
}

// The total of a wave's lanes, in every lane.
template <bool ENT>
__device__ __forceinline__ Total wave_total(Sum q, const Scale &k)
{
    const float m = __builtin_fmaxf(wave_max(q.top), kLowest);
    q.rebase(m, k);
    return Total{m, wave_add(q.s), ENT ? wave_add(q.a) : 0.0f};
}
// The total of NW waves' totals, in every lane: each lane takes one of them (a wave
// that holds a row has few registers to spare).
template <bool ENT, int NW>
__device__ __forceinline__ Total add_waves(const Total *sh, const Scale &k)
{
    auto reduce = [](float x, auto f) {   // over 16 lanes, of which NW hold something
        if constexpr (NW > 1)
            x = f(x, from_lane<kLaneXor1>(x, x));
        if constexpr (NW > 2)
            x = f(x, from_lane<kLaneXor2>(x, x));
        if constexpr (NW > 4)
            x = f(x, from_lane<kMirror8>(x, x));
        if constexpr (NW > 8)
            x = f(x, from_lane<kMirror16>(x, x));
        return x;
    };
    constexpr int M = NW <= 1 ? 1 : NW <= 2 ? 2 : NW <= 4 ? 4 : NW <= 8 ? 8 : 16;
    const int i = threadIdx.x & (M - 1);
    const Total own = i < NW ? sh[i] : Total{kLowest, 0.0f, 0.0f};
    Total t{reduce(own.m, [](float a, float b) { return __builtin_fmaxf(a, b); }), 0.0f, 0.0f};
    add_total(t, own, k);
    t.s = reduce(t.s, [](float a, float b) { return a + b; });
    if constexpr (ENT)
        t.a = reduce(t.a, [](float a, float b) { return a + b; });
    return t;
}
// Every thread gets the workgroup's total.  `sh`: one Total per wave.  One
// barrier; the caller places another before `sh` is written again.
template <bool ENT, int NW = kNW>
__device__ __forceinline__ Total block_total(const Sum &q, const Scale &k, Total *sh)
{
    const Total w = wave_total<ENT>(q, k);
    if ((threadIdx.x & (kWave - 1)) == 0)
        sh[threadIdx.x / kWave] = w;
    __syncthreads();
    return add_waves<ENT, NW>(sh, k);
}

// The total of a row's segments, one workgroup per row, in a fixed order.
__device__ __forceinline__ Total join_parts(const LossPart *p, int segs, const Scale &k, Total *sh)
{
    const int tid = threadIdx.x;
    float m = kLowest;
    for (int i = tid; i < segs; i += kNT)
        m = __builtin_fmaxf(m, p[i].m);
    m = wave_max(m);
    Total t{m, 0.0f, 0.0f};
    for (int i = tid; i < segs; i += kNT)
        add_total(t, Total{p[i].m, p[i].s, p[i].a}, k);
    t.s = wave_add(t.s);
    t.a = wave_add(t.a);
    if ((tid & (kWave - 1)) == 0)
        sh[tid / kWave] = t;
    __syncthreads();
    t = Total{kLowest, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kNW; ++i)
        t.m = __builtin_fmaxf(t.m, sh[i].m);
#pragma unroll
    for (int i = 0; i < kNW; ++i)
        add_total(t, sh[i], k);
    return t;
}

// ln of the sum relative to the exact largest logit, and a token's log
// probability.
__device__ __forceinline__ float ln_sum(const Total &t, const Scale &k)
{
    return kLn2 * (log2f(t.s) - residue(t.m, k));
}
__device__ __forceinline__ float log_prob(float l, const Total &t, float log2s, const Scale &k)
{
    if (__builtin_fabsf(l) > 0x1p100f)   // c l may leave binary32's range where ln p does not
        return (l - t.m) * (k.c * kLn2) - kLn2 * log2s;
    return kLn2 * (rel(l, t.m, t.m * k.c, k) - log2s);
}

// -- rows mapped to gradients ----------------------------------------------------------------

// The gradients of a chunk.
template <typename T, typename F>
__device__ __forceinline__ u32x4 map_chunk(const Chunk<T> &c, F f)
{
    constexpr int W = Chunk<T>::W;
    float x[W], g[W];
    c.widen(x);
#pragma unroll
    for (int i = 0; i < W; ++i)
        g[i] = f(x[i]);
    return pack_chunk<T>(g);
}

// The thread that holds element x of chunks [k0, k0 + n) of a row gone through NT
// at a time from chunk `base` on, or -1.
template <typename T, int NT>
__device__ __forceinline__ int owner_of(const Row<T> &row, int x, int k0, int n, int base)
{
    constexpr int W = Row<T>::W;
    const int at = x + row.phase, k = at / W;
    return k < k0 || k >= k0 + n ? -1 : k < row.full_lo ? at & (W - 1)
           : k < row.full_hi     ? (k - base) % NT : W + (at & (W - 1));
}

// Chunks [k0, k0 + NT U) of a row of logits, U to a thread: read when it is made,
// then mapped to the gradient's row.
template <typename T, int NT, int U>
struct RowPart {
    static constexpr int W = Row<T>::W;
    int lo, hi, e;
    Chunk<T> ch[U];
    float edge;
    __device__ __forceinline__ RowPart(const Row<T> &row, int k0)
        : lo(max(k0, row.full_lo)), hi(min(k0 + NT * U, row.full_hi))
    {
        const int tid = threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (lo + tid + NT * u < hi)
                ch[u].stream(row.chunk(lo + tid + NT * u));
        e = tid < 2 * W ? row.edge(tid, k0, k0 + NT * U) : -1;
        edge = e >= 0 ? row.at(e) : 0.0f;
    }
    // Writes f(logit).
    template <typename F>
    __device__ __forceinline__ void map(const Row<T> &row, T *out, F f) const
    {
        T *first = out + (lo * W - row.phase);
        const bool same = (reinterpret_cast<uintptr_t>(first) & 15) == 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = hi - lo - NT * u;
            if (n <= 0)
                continue;
            const u32x4 g = map_chunk(ch[u], f);
            if (same)
                store_chunks(g, first + NT * W * u, n);
            else if ((int)threadIdx.x < n)
                store_any(g, first + NT * W * u + threadIdx.x * W);
        }
        if (e >= 0)
            store_one(out + e, f(edge));
    }
};

// The same value in every element of chunks [k0, k1), without reading the
// logits.
template <typename T, int NT = kNT>
__device__ __forceinline__ void fill_row(const Row<T> &row, T *out, int k0, int k1, float v)
{
    constexpr int W = Row<T>::W;
    const int lo = max(k0, row.full_lo), hi = min(k1, row.full_hi);
    float g[W];
#pragma unroll
    for (int i = 0; i < W; ++i)
        g[i] = v;
    const u32x4 x = pack_chunk<T>(g);
    for (int k = lo + (int)threadIdx.x; k < hi; k += NT)
        store_any(x, out + (k * W - row.phase));
    const int e = (int)threadIdx.x < 2 * W ? row.edge(threadIdx.x, k0, k1) : -1;
    if (e >= 0)
        store_one(out + e, v);
}

// -- a row held in registers ---------------------------------------------------------------
//
// NT threads of a workgroup hold a row of up to H chunks a thread in their
// registers: the logits are read from memory once, summed as they arrive, and
// turned into gradients from the registers.  The workgroup goes through rows
// gridDim.x apart: once a row's gradients are on their way its registers take the
// next row, so that the loads wait behind the stores and not behind their end.

// Of these, the last chunks a thread parks in LDS once they are summed, which
// leaves registers for what happens between the sums and the gradients (as many
// as the workgroups resident on a compute unit have LDS for).
constexpr int parked(int threads) { return threads >= 448 ? 4 : threads >= 192 ? 2 : 0; }

// SAME: the gradient's rows sit at the 16-byte phase of the logits' rows.
template <typename T, int NT, int H, bool SAME>
struct HeldRow {
    static constexpr int W = Row<T>::W;
    static constexpr int G = 8 / W;       // chunks of a group that is summed at once
    static constexpr int P = parked(NT), P0 = H - P;
    u32x4 *park;  // P NT chunks of LDS
    Row<T> row;
    Chunk<T> ch[H];   // chunk NT i + tid of the row

    float edge;   // this thread's element of the row's partial first or last chunk
    int e;        // and its index, or -1

    __device__ __forceinline__ void take(const Row<T> &next)
    {
        row = next;
        e = (int)threadIdx.x < 2 * W ? next.edge(threadIdx.x, 0, next.chunks) : -1;
        edge = e >= 0 ? next.at(e) : -kInf;
    }
    // Reads a row's whole chunks.  What lies past them is not read.
    __device__ __forceinline__ void read(const Row<T> &next)
    {
        const int m = next.full_hi - next.full_lo;
        const T *first = scalar(next.chunk(next.full_lo));
        const __amdgpu_buffer_rsrc_t rs = window(first, m);
        // threads below full_lo have no first chunk: their offset wraps past the window
        const int at = ((int)threadIdx.x - next.full_lo) * 16;
        int later = at + NT * 16;
        asm volatile("" : "+v"(later));   // in a register: the wrapped sum, not a wrapped offset plus an immediate
#pragma unroll
        for (int i = 0; i < H; ++i)
            ch[i].r = __builtin_bit_cast(decltype(ch[i].r),
                                         __builtin_amdgcn_raw_buffer_load_b128(
                                             rs, i ? later : at, i ? NT * 16 * (i - 1) : 0,
                                             kLoadStreamPolicy));
    }
    // Visits the groups of G chunks that hold anything: f(first chunk, values).
    // Values past the row's whole chunks are -inf, as are those past the H chunks
    // of a thread, where G does not divide H (i + j < H is known once unrolled).
    template <typename F>
    __device__ __forceinline__ void each_group(F f)
    {
#pragma unroll
        for (int i = 0; i < H; i += G) {
            if (NT * i < row.full_hi) {
                float x[W * G];
                u32x4 raw[G];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    if (i + j >= H) {
#pragma unroll
                        for (int w = 0; w < W; ++w)
                            x[j * W + w] = -kInf;
                        continue;
                    }
                    if (i + j == 0 || NT * (i + j + 1) > row.full_hi) {   // kept a branch
                        int t = threadIdx.x;
                        asm volatile("" : "+v"(t));   // or the sums below would be kept over all rows
                        if (t < row.full_lo - NT * (i + j) || t >= row.full_hi - NT * (i + j))
                            ch[i + j].clear();
                    }
                    raw[j] = __builtin_bit_cast(u32x4, ch[i + j].r);
                    float y[W];
                    ch[i + j].widen(y);
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        x[j * W + w] = y[w];
                }
                f(i, x);
#pragma unroll
                for (int j = 0; j < G; ++j)
                    if (i + j >= P0 && i + j < H)
                        park[NT * (i + j - P0) + threadIdx.x] = __builtin_bit_cast(u32x4, raw[j]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // Writes f(logit) for every element the thread holds (nothing unless
    // `write`), then reads `next` (which may be empty) into its place.  `out`: the
    // gradient's row.
    template <typename F>
    __device__ __forceinline__ void map(T *out, bool write, const Row<T> &next, F f)
    {
        T *first = scalar(out - row.phase);   // chunk 0's
        const int hi = write ? row.full_hi : 0;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            Chunk<T> c = ch[i];
            if (i >= P0)
                c.r = __builtin_bit_cast(decltype(c.r), park[NT * (i - P0) + threadIdx.x]);
            else   // opaque, or the widened logits of the sums would be kept from there
                asm volatile("" : "+v"(c.r));
            if constexpr (SAME) {
                const int skip = i ? 0 : row.full_lo;
                if (NT * i < hi)
                    store_chunks(map_chunk(c, f), first + W * (NT * i + skip), hi - NT * i - skip, skip);
            } else {
                if ((int)threadIdx.x < hi - NT * i && (i || (int)threadIdx.x >= row.full_lo))
                    store_any(map_chunk(c, f), first + NT * W * i + threadIdx.x * (unsigned)W);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        read(next);
        if (e >= 0 && write)
            store_one(out + e, f(edge));
    }
};

// -- launches ---------------------------------------------------------------------------------

// Calls f(first row, rows) so that no launch has more than 2^31 threads.
template <typename F>
inline int each_launch(int64_t rows, int per_row, F f, int threads = kNT)
{
    const int64_t most = std::max<int64_t>(1, (int64_t(1) << 31) / threads / per_row);
    for (int64_t r = 0; r < rows; r += most) {
        f(r, (unsigned)std::min(most, rows - r));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// Chunks per workgroup when a row of `vocab` elements at any place in its first
// cache line is cut for `segs` workgroups.
template <typename T>
int chunks_per(int vocab, int segs)
{
    constexpr int W = 16 / (int)sizeof(T), phase = kLine / (int)sizeof(T) - 1;
    const int most = (vocab + phase + W - 1) / W;
    return (most + segs - 1) / segs;
}

// Few rows that are not cut are summed by workgroups of kWide threads.
constexpr int kWide = 1024;
inline bool wide_rows(const LossRows &in) { return in.rows <= kLossWideRows && in.vocab > 4096; }

// Workgroups of a launch that goes through rows: as many as are resident at once
// (128 registers a thread: 16 waves on a compute unit), or one per row where
// each would get four rows or fewer.  Log probabilities, loss and gradient in bf16,
// going through rows and a workgroup per row: 8192 x 128256 (32 rows each) 748 and
// 784 us; 4096 x 50304 (eight) 155 and 147; 2048 x 50304 (four) 82 and 81; 1024 x 50304
// (two) 43 and 46: around the border the two are within 7 %.
inline unsigned held_grid(int64_t rows, int threads)
{
    const int64_t most = (int64_t)device_cu_count() * (1024 / threads);
    return (unsigned)(rows <= 4 * most ? rows : most);
}

// Every row of the gradient starts at its logits' 16-byte phase.
inline bool same_phase(const LossRows &in, const void *d_logits, int64_t d_stride)
{
    const uint64_t es = in.dtype == ZERO_BF16 ? 2 : 4;
    const uint64_t base = (uint64_t)(uintptr_t)in.logits ^ (uint64_t)(uintptr_t)d_logits;
    return base % 16 == 0 && (uint64_t)(in.stride - d_stride) * es % 16 == 0;
}

}  // namespace dev
}  // namespace zero
