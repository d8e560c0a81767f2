// token_loss_kernels.hip -- log probabilities of given tokens (with entropy
// and the top alternatives) and distillation from a teacher's top logits over
// rows of logits, forward and backward.
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
// Bound: HBM.  A forward pass reads each logit once; per bf16 element that is 2
// bytes against 8 to 11 vector issue slots (widen 1, max 1/2, fma 1, exp 4,
// add 1; entropy: clamp 1, fma 1).
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "token_loss.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kNT = kLossBlock;
constexpr int kNW = kNT / kWave;
constexpr float kInf = __builtin_inff();
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLowest = -3.40282346638528859812e38f;
constexpr float kHeadroom = 10.0f;      // binary orders a group may exceed a lane's reference
constexpr float kBig = 0x1p20f;         // |c m| beyond it: t = (l - m) c
constexpr float kTiny = -1000.0f;       // t of a probability that is zero, for products with it

// -- loading -------------------------------------------------------------------------

// 16 bytes of a row: W elements.
template <typename T>
struct Chunk;
template <>
struct Chunk<uint16_t> {
    static constexpr int W = 8;
    u32x4 r;
    __device__ __forceinline__ void load(const uint16_t *p) { r = *reinterpret_cast<const u32x4 *>(p); }
    __device__ __forceinline__ void stream(const uint16_t *p)
    {
        r = ld_stream(reinterpret_cast<const u32x4 *>(p));
    }
    __device__ __forceinline__ void widen(float (&x)[W]) const
    {
        x[0] = bf_lo(r.x), x[1] = bf_hi(r.x), x[2] = bf_lo(r.y), x[3] = bf_hi(r.y);
        x[4] = bf_lo(r.z), x[5] = bf_hi(r.z), x[6] = bf_lo(r.w), x[7] = bf_hi(r.w);
    }
};
template <>
struct Chunk<float> {
    static constexpr int W = 4;
    f32x4 r;
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

// Stores a chunk's gradients, rounded once, at any element alignment (gfx950
// takes 16-byte stores at every address; a row whose gradient sits at another
// 16-byte phase than its logits needs them).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <typename T, int W>
__device__ __forceinline__ void store_chunk(T *p, const float (&g)[W])
{
    u32x4 v;
    if constexpr (sizeof(T) == 2)
        v = u32x4{pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]),
                  pack_bf16x2(g[6], g[7])};
    else
        v = u32x4{__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]),
                  __float_as_uint(g[3])};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any *>(p));
}
__device__ __forceinline__ void store_one(uint16_t *p, float g) { *p = to_bf16(g); }
__device__ __forceinline__ void store_one(float *p, float g) { *p = g; }

// A row cut into chunks that start at 16-byte boundaries: chunk k holds
// elements k W - phase .. + W - 1, whole for full_lo <= k < full_hi; the first
// and last may stick out of the row and are read element by element.
template <typename T>
struct Row {
    static constexpr int W = Chunk<T>::W;
    const T *p;
    int vocab, phase, chunks, full_lo, full_hi;
    __device__ __forceinline__ Row(const void *base, int64_t off, int vocab_) : vocab(vocab_)
    {
        p = static_cast<const T *>(base) + off;
        phase = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
        chunks = (vocab + phase + W - 1) / W;
        full_lo = phase ? 1 : 0;
        full_hi = max(full_lo, (vocab + phase) / W);
    }
    __device__ __forceinline__ const T *chunk(int k) const { return p + ((int64_t)k * W - phase); }
    __device__ __forceinline__ float at(int e) const { return grad_at<T>(p, e); }
    // Element of edge slot s (0 .. 2W-1: the head's, then the tail's) among
    // chunks [k0, k1), or -1.
    __device__ __forceinline__ int edge(int s, int k0, int k1) const
    {
        const int k = s < W ? 0 : full_hi;
        const int e = k * W - phase + (s & (W - 1));
        const bool partial = s < W ? full_lo == 1 : full_hi < chunks;
        return partial && k >= k0 && k < k1 && e >= 0 && e < vocab ? e : -1;
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
// t of reference m against reference n, as the sums were formed.
__device__ __forceinline__ float shift_of(float m, float n, const Scale &k)
{
    return __builtin_fabsf(m) > k.big || __builtin_fabsf(n) > k.big ? (m - n) * k.c : m * k.c - n * k.c;
}
// c m - fl(c m): what the sums' reference R is off the exact one by.
__device__ __forceinline__ float residue(float m, const Scale &k)
{
    return __builtin_fabsf(m) > k.big ? 0.0f : __builtin_fmaf(m, k.c, -(m * k.c));
}
__device__ __forceinline__ float pow2(float t) { return __builtin_amdgcn_exp2f(t); }

struct Sum {
    float top;       // the largest logit seen
    float m, r;      // the reference and fl(c m)
    float thr;       // groups whose largest logit is above it raise the reference
    float s, a;      // sums of 2^t and of t 2^t
    __device__ __forceinline__ Sum() : top(-kInf), m(kLowest), r(0), thr(kLowest), s(0), a(0) {}

    __device__ __forceinline__ void rebase(float n, const Scale &k)
    {
        const float d = shift_of(m, n, k), f = pow2(d);
        a = f * (a + __builtin_fmaxf(d, kTiny) * s);
        s = s * f;
        m = n;
        r = n * k.c;
    }

    // Adds N elements.  A NaN among them makes the sum NaN (max ignores it).
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
        if (g > thr) {
            rebase(g, k);
            thr = g + k.gap;
        }
        if (__any(__builtin_fabsf(m) > k.big))
            add_terms<N, ENT, true>(x, k);
        else
            add_terms<N, ENT, false>(x, k);
    }
    template <int N, bool ENT, bool BIG>
    __device__ __forceinline__ void add_terms(const float (&x)[N], const Scale &k)
    {
        // a group's sums apart from the lane's: shorter chains round less
        float sg = 0, ag = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = BIG ? rel(x[i], m, r, k) : __builtin_fmaf(x[i], k.c, -r);
            const float e = pow2(t);
            sg += e;
            if constexpr (ENT)
                ag = __builtin_fmaf(e, __builtin_fmaxf(t, kTiny), ag);
        }
        s += sg;
        if constexpr (ENT)
            a += ag;
    }
};

// The sum of a wave's or workgroup's lanes against the largest logit among
// them (kLowest at least), in a fixed order.
struct Total {
    float m, s, a;
    __device__ __forceinline__ bool empty() const { return s == 0.0f; }   // every logit -inf
};

__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        x = __builtin_fmaxf(x, __shfl_xor(x, o, kWave));
    return x;
}
__device__ __forceinline__ float wave_add(float x)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        x += __shfl_xor(x, o, kWave);
    return x;
}

// One of several totals moved to reference m and added.
__device__ __forceinline__ void add_total(Total &t, const Total &o, const Scale &k)
{
    const float d = shift_of(o.m, t.m, k), f = pow2(d);
    t.a += f * (o.a + __builtin_fmaxf(d, kTiny) * o.s);
    t.s += f * o.s;
}

// Every thread gets the workgroup's total.  `sh`: one Total per wave.  One
// barrier; the caller places another before `sh` is written again.
template <bool ENT, int NW = kNW>
__device__ __forceinline__ Total block_total(Sum q, const Scale &k, Total *sh)
{
    const float m = __builtin_fmaxf(wave_max(q.top), kLowest);
    q.rebase(m, k);
    Total w{m, wave_add(q.s), ENT ? wave_add(q.a) : 0.0f};
    if ((threadIdx.x & (kWave - 1)) == 0)
        sh[threadIdx.x / kWave] = w;
    __syncthreads();
    Total t{kLowest, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NW; ++i)
        t.m = __builtin_fmaxf(t.m, sh[i].m);
#pragma unroll
    for (int i = 0; i < NW; ++i)
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

// -- selection -----------------------------------------------------------------------------
//
// The K largest logits, ties to the lowest index, as keys that order them: the
// logit's bits made monotonic, then the inverted index.  One pass over the row
// leaves the largest logit of each of at most kGroups groups of a few chunks in
// LDS.  The K-th largest of those is at most the K-th largest logit, so only
// groups that reach it are read again (about K of them) and their logits that
// reach it become candidates, usually little more than K.  Where there are too
// many (plateaus of equal logits), a radix search over the whole keys, which are
// all different, finds the K-th exactly.

constexpr int kIndexBits = 20;
static_assert(ZERO_MAX_VOCAB <= 1 << kIndexBits, "the index fits its field");
constexpr int kGroups = 2048;
constexpr int kCands = 1024;

__device__ __forceinline__ unsigned ord32(float x)
{
    const unsigned u = __float_as_uint(x + 0.0f);   // -0 -> +0
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float ord32_value(unsigned k)
{
    return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, int index)
{
    return (uint64_t)ord32(x) << kIndexBits | (unsigned)((1 << kIndexBits) - 1 - index);
}
__device__ __forceinline__ float key_value(uint64_t k) { return ord32_value((unsigned)(k >> kIndexBits)); }
__device__ __forceinline__ int key_index(uint64_t k)
{
    return (1 << kIndexBits) - 1 - (int)(k & ((1 << kIndexBits) - 1));
}

struct Select {
    unsigned hist[256];
    unsigned count;        // candidates
    unsigned listed;       // groups to read again
    unsigned bin, above;   // a radix pass's result
    float gmax[kGroups];
    uint16_t list[kGroups];
    uint64_t cand[kCands];
};

// One radix pass's choice: the bin of sh.hist (256 bins) that holds the want-th
// largest entry, and how many lie above it.  Thread b owns bin b.
__device__ __forceinline__ void pick_bin(Select &sh, unsigned want)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    __syncthreads();
    const unsigned own = sh.hist[tid];
    unsigned above = 0;                     // entries in bins above this one
    for (int w = wave + 1; w < kNW; ++w)
        above += sh.hist[w * kWave + lane];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        above += __shfl_xor(above, o, kWave);
    unsigned suf = own;                     // of this wave: inclusive suffix sum
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const unsigned v = __shfl_down(suf, o, kWave);
        suf += lane + o < kWave ? v : 0;
    }
    above += suf - own;
    if (above < want && above + own >= want) {
        sh.bin = tid;
        sh.above = above;
    }
    __syncthreads();
}

// Adds one to hist[bin] for every active lane; a wave that agrees on the bin
// does so with one addition (plateaus would serialize otherwise).
__device__ __forceinline__ void count_bin(Select &sh, unsigned bin)
{
    const unsigned first = __builtin_amdgcn_readfirstlane(bin);
    const uint64_t act = __ballot(1), same = __ballot(bin == first);
    if (act == same) {
        if ((int)__builtin_ctzll(act) == (int)(threadIdx.x & (kWave - 1)))
            atomicAdd(&sh.hist[first], (unsigned)__popcll(act));
    } else {
        atomicAdd(&sh.hist[bin], 1u);
    }
}

// The K-th largest of the keys that `each` visits (all different, at least K of
// them).  each(f) calls f(key) once for every key, over the whole workgroup.
template <typename Each>
__device__ uint64_t kth_key(Select &sh, int K, Each each)
{
    uint64_t prefix = 0;
    unsigned want = (unsigned)K;
    for (int sft = 48; sft >= 0; sft -= 8) {   // 32 + 20 bits in seven bytes
        sh.hist[threadIdx.x] = 0;
        __syncthreads();
        each([&](uint64_t k) {
            if ((k >> sft) >> 8 == prefix)
                count_bin(sh, (unsigned)(k >> sft) & 255u);
        });
        pick_bin(sh, want);
        prefix = prefix << 8 | sh.bin;
        want -= sh.above;
        __syncthreads();
    }
    return prefix;
}

__device__ __forceinline__ void push(Select &sh, uint64_t key)
{
    const unsigned at = atomicAdd(&sh.count, 1u);
    if (at < (unsigned)kCands)
        sh.cand[at] = key;
}

// Visits the elements of chunks [k0, k1) of a row: f(value, index).
template <typename T, typename F>
__device__ __forceinline__ void each_element(const Row<T> &row, int k0, int k1, F f)
{
    constexpr int W = Row<T>::W;
    const int lo = max(k0, row.full_lo), hi = min(k1, row.full_hi);
    for (int k = lo + (int)threadIdx.x; k < hi; k += kNT) {
        Chunk<T> ch;
        ch.load(row.chunk(k));
        float x[W];
        ch.widen(x);
#pragma unroll
        for (int i = 0; i < W; ++i)
            f(x[i], k * W - row.phase + i);
    }
    const int e = (int)threadIdx.x < 2 * W ? row.edge(threadIdx.x, k0, k1) : -1;
    if (e >= 0)
        f(row.at(e), e);
}

// Writes the K largest of the workgroup's candidates, best first, through
// put(rank, key).  Every candidate's rank is the number of larger ones.
template <typename Put>
__device__ __forceinline__ void put_ranked(Select &sh, int n, int K, Put put)
{
    for (int i = threadIdx.x; i < n; i += kNT) {
        const uint64_t own = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j)
            rank += sh.cand[j] > own;
        if (rank < K)
            put(rank, own);
    }
}

// The K largest logits of chunks [k0, k1), whose groups' largest logits are in
// sh.gmax: group g = thread + kNT * (batch / per), a batch being the U chunks
// lo + thread + kNT * (batch * U + u).
template <typename T, int U, typename Put>
__device__ void select_top(Select &sh, const Row<T> &row, int k0, int k1, int groups, int per, int K,
                           Put put)
{
    constexpr int W = Row<T>::W;
    const int tid = threadIdx.x;
    const int lo = max(k0, row.full_lo), hi = min(k1, row.full_hi);
    const int first = max(k0 * W - row.phase, 0), last = min(k1 * W - row.phase, row.vocab);
    const int n = max(last - first, 0);
    // the K-th largest group maximum, to 16 bits (a lower bound of it)
    unsigned floor16 = 0;
    if (groups >= K) {
        unsigned want = (unsigned)K;
        for (int pass = 0; pass < 2; ++pass) {
            sh.hist[tid] = 0;
            __syncthreads();
            for (int g = tid; g < groups; g += kNT) {
                const unsigned o = ord32(sh.gmax[g]);
                if (pass == 0)
                    count_bin(sh, o >> 24);
                else if (o >> 24 == floor16)
                    count_bin(sh, o >> 16 & 255u);
            }
            pick_bin(sh, want);
            floor16 = floor16 << 8 | sh.bin;
            want -= sh.above;
            __syncthreads();
        }
    }
    const uint64_t bound = (uint64_t)(floor16 << 16) << kIndexBits;
    if (tid == 0) {
        sh.count = 0;
        sh.listed = 0;
    }
    __syncthreads();
    for (int g = tid; g < groups; g += kNT)
        if (ord32(sh.gmax[g]) >> 16 >= floor16)
            sh.list[atomicAdd(&sh.listed, 1u)] = (uint16_t)g;
    __syncthreads();
    const int span = per * U;
    const int todo = (int)sh.listed * span;
    for (int j = tid; j < todo; j += kNT) {
        const int g = sh.list[j / span], step = (g / kNT) * span + j % span;
        const int k = lo + (g % kNT) + kNT * step;
        if (k < hi) {
            Chunk<T> ch;
            ch.load(row.chunk(k));
            float x[W];
            ch.widen(x);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint64_t key = key_of(x[i], k * W - row.phase + i);
                if (key >= bound)
                    push(sh, key);
            }
        }
    }
    const int e = tid < 2 * W ? row.edge(tid, k0, k1) : -1;
    if (e >= 0) {
        const uint64_t key = key_of(row.at(e), e);
        if (key >= bound)
            push(sh, key);
    }
    __syncthreads();
    int cands = (int)sh.count;
    if (cands > kCands) {
        __syncthreads();
        uint64_t kth = 0;
        if (n > K)
            kth = kth_key(sh, K, [&](auto f) {
                each_element(row, k0, k1, [&](float x, int i) { f(key_of(x, i)); });
            });
        if (tid == 0)
            sh.count = 0;
        __syncthreads();
        each_element(row, k0, k1, [&](float x, int i) {
            const uint64_t key = key_of(x, i);
            if (key >= kth)
                push(sh, key);
        });
        __syncthreads();
        cands = min((int)sh.count, kCands);
    }
    put_ranked(sh, cands, K, put);
}

// -- log probabilities: forward ----------------------------------------------------------

// A row's outputs from its total and the given token's logit (anything where
// the token is outside the vocabulary); the top alternatives go out separately.
__device__ __forceinline__ void finish_logprob(const LogprobArgs &a, int64_t row, float l, const Total &t)
{
    if (threadIdx.x != 0)
        return;
    const Scale k(a.in.c);
    const bool none = t.empty();
    const float log2s = log2f(t.s);
    if (a.stats) {
        a.stats[2 * row] = none ? -kInf : t.m;
        a.stats[2 * row + 1] = none ? -kInf : ln_sum(t, k);
    }
    if (a.entropy) {
        const float h = kLn2 * (log2s - t.a / t.s);
        a.entropy[row] = none || h < 0.0f ? 0.0f : h;
    }
    if (a.logprob) {
        a.logprob[row] = a.tokens[row] >= a.in.vocab ? __builtin_nanf("")
                         : none                      ? -kInf
                                                     : log_prob(l, t, log2s, k);
    }
}

// The logit of a row's given token; 0 where there is none in the vocabulary.
template <typename T>
__device__ __forceinline__ float token_logit(const LogprobArgs &a, int64_t row)
{
    const int64_t tok = a.tokens ? a.tokens[row] : -1;
    return tok >= 0 && tok < a.in.vocab
               ? grad_at<T>(static_cast<const T *>(a.in.logits) + row * a.in.stride, tok) : 0.0f;
}

// What a padding row (a negative token) leaves: zeros, no alternatives.
__device__ __forceinline__ void pad_logprob(const LogprobArgs &a, int64_t row)
{
    if (threadIdx.x == 0) {
        if (a.stats)
            a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
        if (a.entropy)
            a.entropy[row] = 0.0f;
        if (a.logprob)
            a.logprob[row] = 0.0f;
    }
    for (int i = threadIdx.x; i < a.top_k; i += blockDim.x) {
        a.top_index[row * a.top_k + i] = -1;
        a.top_logprob[row * a.top_k + i] = -kInf;
    }
}

__device__ __forceinline__ void put_top(const LogprobArgs &a, int64_t row, int rank, uint64_t key,
                                        const Total &t, float log2s)
{
    const float l = key_value(key);
    a.top_index[row * a.top_k + rank] = l == -kInf ? -1 : key_index(key);
    a.top_logprob[row * a.top_k + rank] = l == -kInf ? -kInf : log_prob(l, t, log2s, Scale(a.in.c));
}
__device__ __forceinline__ void put_none(const LogprobArgs &a, int64_t row, int from, const Total &t)
{
    for (int i = from + (int)threadIdx.x; i < a.top_k; i += kNT) {
        a.top_index[row * a.top_k + i] = -1;
        a.top_logprob[row * a.top_k + i] = t.s != t.s ? __builtin_nanf("") : -kInf;
    }
}

// One workgroup per segment of a row (segs of them): the whole result where
// segs is 1, else its LossPart and its top keys.
template <typename T, bool ENT, bool TOP>
__global__ __launch_bounds__(kNT) void logprob_kernel(LogprobArgs a, int64_t row0, int segs, int cps)
{
    constexpr int U = 4, W = Row<T>::W;
    __shared__ Total tot[kNW];
    __shared__ typename std::conditional<TOP, Select, int>::type sh;
    const int64_t row_i = row0 + blockIdx.x / segs;
    const int seg = blockIdx.x % segs, tid = threadIdx.x;
    if (a.tokens && a.tokens[row_i] < 0) {
        if (segs == 1)
            pad_logprob(a, row_i);
        return;
    }
    const Row<T> row(a.in.logits, row_i * a.in.stride, a.in.vocab);
    const int k0 = min(seg * cps, row.chunks), k1 = min(k0 + cps, row.chunks);
    const int lo = max(k0, row.full_lo), hi = min(k1, row.full_hi);
    const Scale sc(a.in.c);
    Sum q;
    const int batches = hi > lo ? (hi - lo + kNT * U - 1) / (kNT * U) : 0;
    const int per = (batches + kGroups / kNT - 1) / (kGroups / kNT);   // batches per group
    int in_group = 0, group = tid;
    float gm = -kInf;
    for (int b = 0; b < batches; ++b) {
        const int k = lo + tid + kNT * U * b;
        float g = -kInf;
        if (k + kNT * (U - 1) < hi) {
            Chunk<T> ch[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                ch[u].stream(row.chunk(k + kNT * u));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[W];
                ch[u].widen(x);
                float m = x[0];
#pragma unroll
                for (int i = 1; i < W; ++i)
                    m = __builtin_fmaxf(m, x[i]);
                q.add_with_max<W, ENT>(x, m, sc);
                g = __builtin_fmaxf(g, m);
            }
        } else {
            for (int kk = k; kk < hi; kk += kNT) {
                Chunk<T> ch;
                ch.stream(row.chunk(kk));
                float x[W];
                ch.widen(x);
                float m = x[0];
#pragma unroll
                for (int i = 1; i < W; ++i)
                    m = __builtin_fmaxf(m, x[i]);
                q.add_with_max<W, ENT>(x, m, sc);
                g = __builtin_fmaxf(g, m);
            }
        }
        if constexpr (TOP) {
            gm = __builtin_fmaxf(gm, g);
            if (++in_group == per || b + 1 == batches) {
                sh.gmax[group] = gm;
                gm = -kInf;
                group += kNT;
                in_group = 0;
            }
        }
    }
    const int e = tid < 2 * W ? row.edge(tid, k0, k1) : -1;
    if (e >= 0) {
        const float x[1] = {row.at(e)};
        q.add<1, ENT>(x, sc);
    }
    const Total t = block_total<ENT>(q, sc, tot);
    if (segs == 1)
        finish_logprob(a, row_i, token_logit<T>(a, row_i), t);
    else if (tid == 0)
        a.parts[row_i * segs + seg] = LossPart{t.m, t.s, t.a, 0.0f};
    if constexpr (TOP) {
        const int groups = per ? (batches + per - 1) / per * kNT : 0;
        const int n = max(min(k1 * W - row.phase, row.vocab) - max(k0 * W - row.phase, 0), 0);
        __syncthreads();
        if (t.s != t.s) {   // a NaN or +inf logit: no order, no alternatives
            if (segs == 1)
                put_none(a, row_i, 0, t);
        } else if (segs == 1) {
            const float log2s = log2f(t.s);
            select_top<T, U>(sh, row, k0, k1, groups, per, a.top_k,
                             [&](int r, uint64_t key) { put_top(a, row_i, r, key, t, log2s); });
            put_none(a, row_i, n, t);
        } else {
            uint64_t *out = a.keys + (row_i * segs + seg) * a.top_k;
            select_top<T, U>(sh, row, k0, k1, groups, per, a.top_k,
                             [&](int r, uint64_t key) { out[r] = key; });
            for (int i = n + tid; i < a.top_k; i += kNT)
                out[i] = 0;   // below every logit's key
        }
    }
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

template <bool TOP>
__global__ __launch_bounds__(kNT) void logprob_join_kernel(LogprobArgs a, int64_t row0, int segs)
{
    __shared__ Total tot[kNW];
    __shared__ typename std::conditional<TOP, Select, int>::type sh;
    const int64_t row = row0 + blockIdx.x;
    const int tid = threadIdx.x;
    if (a.tokens && a.tokens[row] < 0) {
        pad_logprob(a, row);
        return;
    }
    const Total t = join_parts(a.parts + row * segs, segs, Scale(a.in.c), tot);
    finish_logprob(a, row, a.in.dtype == ZERO_BF16 ? token_logit<uint16_t>(a, row)
                                                   : token_logit<float>(a, row), t);
    if constexpr (TOP) {
        if (t.s != t.s) {
            put_none(a, row, 0, t);
            return;
        }
        const uint64_t *keys = a.keys + row * segs * a.top_k;
        const int n = segs * a.top_k;
        const float log2s = log2f(t.s);
        if (tid == 0)
            sh.count = 0;
        __syncthreads();
        uint64_t least = 1;   // absent alternatives are zero keys
        if (n > kCands) {
            // at least K keys are not zero where the row has K logits; if it has
            // fewer, the K-th is zero and every key that is not stays
            least = kth_key(sh, a.top_k, [&](auto f) {
                for (int i = tid; i < n; i += kNT)
                    f(keys[i]);
            });
            if (least == 0)
                least = 1;
        }
        for (int i = tid; i < n; i += kNT) {
            const uint64_t k = keys[i];
            if (k >= least)
                push(sh, k);
        }
        __syncthreads();
        const int cands = min((int)sh.count, kCands);
        put_ranked(sh, cands, a.top_k,
                   [&](int r, uint64_t key) { put_top(a, row, r, key, t, log2s); });
        put_none(a, row, cands, t);
    }
}

// -- gradients ------------------------------------------------------------------------------

// Visits chunks [k0, k1) of a row of logits and writes what f(logit) returns to
// the same elements of the gradient's row; element `hot` gets `add` more.
template <typename T, typename F>
__device__ __forceinline__ void map_row(const Row<T> &row, T *out, int k0, int k1, int hot, float add,
                                        F f)
{
    constexpr int W = Row<T>::W;
    const int tid = threadIdx.x;
    const int lo = max(k0, row.full_lo), hi = min(k1, row.full_hi);
    const int hot_k = hot < 0 ? -1 : (hot + row.phase) / W, hot_i = (hot + row.phase) & (W - 1);
    for (int k = lo + tid; k < hi; k += kNT) {
        Chunk<T> ch;
        ch.stream(row.chunk(k));
        float x[W], g[W];
        ch.widen(x);
#pragma unroll
        for (int i = 0; i < W; ++i)
            g[i] = f(x[i]);
        if (k == hot_k) {
#pragma unroll
            for (int i = 0; i < W; ++i)
                g[i] = i == hot_i ? g[i] + add : g[i];
        }
        store_chunk(out + (k * W - row.phase), g);
    }
    const int e = tid < 2 * W ? row.edge(tid, k0, k1) : -1;
    if (e >= 0) {
        const float g = f(row.at(e));
        store_one(out + e, e == hot ? g + add : g);
    }
}

// The same value in every element, without reading the logits.
template <typename T, int NT = kNT>
__device__ __forceinline__ void fill_row(const Row<T> &row, T *out, int k0, int k1, float v)
{
    constexpr int W = Row<T>::W;
    const int lo = max(k0, row.full_lo), hi = min(k1, row.full_hi);
    float g[W];
#pragma unroll
    for (int i = 0; i < W; ++i)
        g[i] = v;
    for (int k = lo + (int)threadIdx.x; k < hi; k += NT)
        store_chunk(out + (k * W - row.phase), g);
    const int e = (int)threadIdx.x < 2 * W ? row.edge(threadIdx.x, k0, k1) : -1;
    if (e >= 0)
        store_one(out + e, v);
}

// d_logits_j = scale (d_lp ([j = t] - p_j) - d_H p_j (ln p_j + H)).  With p_j =
// 2^t inv this is [j = t] scale d_lp - p_j (u + v t), u and v the row's.
template <typename T, bool ENT>
__global__ __launch_bounds__(kNT) void logprob_grad_kernel(LogprobGradArgs a, int64_t row0, int segs,
                                                           int cps)
{
    const int64_t r = row0 + blockIdx.x / segs;
    const int seg = blockIdx.x % segs;
    const Row<T> row(a.in.logits, r * a.in.stride, a.in.vocab);
    T *out = static_cast<T *>(a.d_logits) + r * a.d_stride;
    const int k0 = min(seg * cps, row.chunks), k1 = min(k0 + cps, row.chunks);
    const int64_t tok = a.tokens ? a.tokens[r] : 0;
    const float dl = a.d_logprob ? a.d_logprob[r] : 0.0f;
    const float dh = ENT ? a.d_entropy[r] : 0.0f;
    const float m = a.stats[2 * r], ln = a.stats[2 * r + 1];
    const bool zero = tok < 0 || (dl == 0.0f && dh == 0.0f), bad = tok >= a.in.vocab;
    if (zero || bad || m == -kInf) {
        fill_row(row, out, k0, k1, bad && !zero ? __builtin_nanf("") : 0.0f);
        return;
    }
    const Scale k(a.in.c);
    const float c = k.c, ref = m * c;
    // log2 p = t - off
    const float off = residue(m, k) + ln * 1.44269504088896340736f;
    const float inv = pow2(-off);
    const float h = ENT ? a.entropy[r] : 0.0f;
    const float u = a.in.scale * (dl + dh * (h - off * kLn2)) * inv;
    const float v = a.in.scale * dh * kLn2 * inv;
    const int hot = a.d_logprob ? (int)tok : -1;
    const float add = a.in.scale * dl;
    auto grad = [&](float t) {
        return pow2(t) * (ENT ? __builtin_fmaf(-v, __builtin_fmaxf(t, kTiny), -u) : -u);
    };
    if (__builtin_fabsf(m) > k.big)
        map_row(row, out, k0, k1, hot, add, [&](float x) { return grad((x - m) * c); });
    else
        map_row(row, out, k0, k1, hot, add, [&](float x) { return grad(__builtin_fmaf(x, c, -ref)); });
}

// -- distillation ------------------------------------------------------------------------------

// The teacher's record of a row, as one wave leaves it in LDS.  Entry k of the
// record is lane k % 64's.  binary64 throughout: 1 - sum q would lose the rest's
// digits in binary32.
constexpr int kTopLane = ZERO_MAX_TOP / kWave;   // entries a lane holds at most
struct Teacher {
    double q[ZERO_MAX_TOP], log_q[ZERO_MAX_TOP];
    double token_q[ZERO_MAX_TOP];   // the token's probability over all entries that name it
    double total, rest;             // sum of q and rest; the other tokens' probability
    double max, ln;                 // of the row's logits: largest, ln of the sum relative to it
    double listed_max, listed_sum;  // of the listed tokens, each once
    alignas(16) int index[ZERO_MAX_TOP];   // the token; -1: no token of the vocabulary
    int lead[ZERO_MAX_TOP];         // the token where this is the first entry that names it, else -1
    float logit[ZERO_MAX_TOP];      // the student's
    int any, bad;                   // an entry at all; one outside the vocabulary or with a NaN value
};

// Orders a wave's LDS writes before its lanes' later reads.
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
__device__ __forceinline__ double wave_max_f64(double x)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        x = fmax(x, __shfl_xor(x, o, kWave));
    return x;
}

// Below this the rest's probability is the rounding of the listed ones: binary32
// log probabilities v put at most |v| 2^-24 into each exp(v), and sum q |v| is
// an entropy, below 16 nats for any vocabulary here.
constexpr double kLeastRest = 0x1p-20;

// True (for every lane) where a record is padding: no entry, and no NaN value.
__device__ __forceinline__ bool is_padding(const int32_t *index, const float *value, int K, int lane)
{
    bool some = false;
    for (int k = lane; k < K; k += kWave) {
        const float v = value[k];
        some = some || index[k] >= 0 || v != v;
    }
    return !__any(some);
}

// Reads a row's record (one whole wave calls it).
__device__ __forceinline__ void read_teacher(Teacher &te, const int32_t *index, const float *value,
                                             int K, int mode, int vocab, int lane)
{
    int id[kTopLane];
    double v[kTopLane];
    bool some = false, bad = false;
#pragma unroll
    for (int j = 0; j < kTopLane; ++j) {
        const int k = lane + kWave * j;
        id[j] = k < K ? index[k] : -1;
        const float val = k < K ? value[k] : 0.0f;
        const bool nan = val != val;
        some = some || id[j] >= 0 || nan;
        bad = bad || id[j] >= vocab || nan;
        if (id[j] >= vocab)
            id[j] = -1;
        id[j] = id[j] < 0 ? -1 : id[j];
        v[j] = id[j] >= 0 ? (double)val : -__builtin_inf();
        te.index[k] = id[j];
    }
    some = __any(some);
    bad = __any(bad);
    // q: exp of the given value, or the softmax over the entries
    const bool renorm = mode == ZERO_DISTILL_RENORM;
    double top = -1e300, sum = 0.0;
#pragma unroll
    for (int j = 0; j < kTopLane; ++j)
        top = fmax(top, v[j]);
    top = renorm ? wave_max_f64(top) : 0.0;
    double q[kTopLane];
#pragma unroll
    for (int j = 0; j < kTopLane; ++j) {
        q[j] = id[j] >= 0 ? exp(v[j] - top) : 0.0;
        sum += q[j];
    }
    sum = wave_sum(sum);
    double total, rest = 0.0;
    if (renorm) {
        const double ln = log(sum);
#pragma unroll
        for (int j = 0; j < kTopLane; ++j) {
            q[j] = sum == 0.0 ? 0.0 : q[j] / sum;   // no finite value at all: no distribution
            v[j] = v[j] - top - ln;
        }
        total = sum != sum ? sum : sum == 0.0 ? 0.0 : 1.0;
    } else {
        rest = 1.0 - sum;
        if (rest < kLeastRest)
            rest = 0.0;
        total = sum + rest;
    }
    // entries that name the same token: the first of them stands for it
    int same[kTopLane] = {}, named = 0;
    wave_sync();
    for (int k = 0; k < K; k += 4) {
        const int4 o = *reinterpret_cast<const int4 *>(&te.index[k]);
#pragma unroll
        for (int j = 0; j < kTopLane; ++j)
            same[j] += (o.x == id[j]) + (o.y == id[j]) + (o.z == id[j]) + (o.w == id[j]);
    }
    bool twice = false;
#pragma unroll
    for (int j = 0; j < kTopLane; ++j) {
        const int k = lane + kWave * j;
        te.q[k] = te.token_q[k] = q[j];
        te.log_q[k] = v[j];
        te.lead[k] = id[j];
        twice = twice || (id[j] >= 0 && same[j] > 1);
    }
    if (__any(twice)) {
        wave_sync();
#pragma unroll
        for (int j = 0; j < kTopLane; ++j) {
            if (id[j] < 0 || same[j] < 2)
                continue;
            const int k = lane + kWave * j;
            double sq = 0.0;
            for (int o = 0; o < K; ++o)
                if (te.index[o] == id[j]) {
                    sq += te.q[o];
                    if (o < k)
                        te.lead[k] = -1;
                }
            te.token_q[k] = sq;
        }
        wave_sync();
    }
#pragma unroll
    for (int j = 0; j < kTopLane; ++j)
        named += __popcll(__ballot(te.lead[lane + kWave * j] >= 0));
    if (named == vocab && rest != 0.0) {   // no token is left for the rest
        total -= rest;
        rest = 0.0;
    }
    if (lane == 0) {
        te.total = total;
        te.rest = rest;
        te.any = some;
        te.bad = bad;
    }
}

// The listed tokens' logits and their part of the row's sum (one whole wave,
// after read_teacher).
template <typename T>
__device__ __forceinline__ void read_listed(Teacher &te, const T *p, double scale, int lane)
{
    double l[kTopLane], m = -__builtin_inf(), s = 0.0;
    bool lead[kTopLane];
#pragma unroll
    for (int j = 0; j < kTopLane; ++j) {
        const int k = lane + kWave * j, id = te.index[k];
        const float x = id >= 0 ? grad_at<T>(p, id) : 0.0f;
        lead[j] = te.lead[k] >= 0;
        te.logit[k] = x;
        l[j] = lead[j] ? (double)x : -__builtin_inf();
        m = fmax(m, l[j]);
    }
    m = wave_max_f64(m);
    const double ref = fmax(m, (double)kLowest);
#pragma unroll
    for (int j = 0; j < kTopLane; ++j)
        s += lead[j] ? exp((l[j] - ref) * scale) : 0.0;
    s = wave_sum(s);
    if (lane == 0) {
        te.listed_max = m;
        te.listed_sum = s;
    }
}

// The row's loss and statistics from the total over the tokens that are not
// listed (one whole wave, after read_listed).
__device__ __forceinline__ void finish_distill(Teacher &te, const Total &tail, int K,
                                               const LossRows &in, float *loss, float *stats,
                                               int64_t row, int lane)
{
    const double scale = (double)in.scale;
    const bool tail_none = tail.empty();
    const double tm = tail_none ? -__builtin_inf() : (double)tail.m;
    const double tail_ln = tail_none ? -__builtin_inf() : (double)ln_sum(tail, Scale(in.c));
    wave_sync();
    const double lm = te.listed_max, m = fmax(lm, tm), ref = fmax(m, (double)kLowest);
    const double ls = te.listed_sum * exp((fmax(lm, (double)kLowest) - ref) * scale);
    const double tail_s = tail_none ? 0.0 : exp((tm - ref) * scale + tail_ln);
    const double ln = log(ls + tail_s);
    const bool none = ls + tail_s == 0.0;
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < kTopLane; ++j) {
        const int k = lane + kWave * j;
        if (k < K) {
            const double q = te.q[k];
            const double lp = none ? -__builtin_inf() : ((double)te.logit[k] - ref) * scale - ln;
            if (q != 0.0)   // NaN too
                sum += q * (te.log_q[k] - lp);
        }
    }
    sum = wave_sum(sum);
    const double rest = te.rest;
    if (rest > 0.0) {
        const double lp = none || tail_none ? -__builtin_inf() : (tm - ref) * scale + tail_ln - ln;
        sum += rest * (log(rest) - lp);
    }
    if (lane == 0) {
        te.max = m;
        te.ln = ln;
        if (loss)
            loss[row] = te.bad ? __builtin_nanf("") : (float)sum;
        if (stats) {
            stats[4 * row] = none ? -kInf : (float)m;
            stats[4 * row + 1] = none ? -kInf : (float)ln;
            stats[4 * row + 2] = (float)tm;
            stats[4 * row + 3] = (float)tail_ln;
        }
    }
}
__device__ __forceinline__ void pad_distill(float *loss, float *stats, int64_t row)
{
    if (threadIdx.x == 0) {
        if (loss)
            loss[row] = 0.0f;
        if (stats)
            stats[4 * row] = stats[4 * row + 1] = stats[4 * row + 2] = stats[4 * row + 3] = 0.0f;
    }
}

// A listed token's gradient, entry k's.
__device__ __forceinline__ float listed_grad(const Teacher &te, int k, double m, double ln, double w,
                                             double scale)
{
    const double p = exp(((double)te.logit[k] - m) * scale - ln);
    return (float)(w * (te.total * p - te.token_q[k]));
}

// Marks the listed tokens of chunks [k0, k1) in `bits`, one bit per element of
// the chunks (one whole wave).
__device__ __forceinline__ void mark_listed(unsigned *bits, int words, const int32_t *index, int K,
                                            int base, int end, int vocab, int lane)
{
    for (int i = lane; i < words; i += kWave)
        bits[i] = 0;
    wave_sync();
    for (int k = lane; k < K; k += kWave) {
        const int id = index[k], at = id + base;
        if (id >= 0 && id < vocab && at >= 0 && at < end)
            atomicOr(&bits[at >> 5], 1u << (at & 31));
    }
}

// Words of a segment's bitmap: one bit per element of its chunks, whose first
// and last may stick out of it.
constexpr int kBitWords = (int)(kLossMaxSegment / 32) + 8;

// One workgroup per segment of a row: the sum over its tokens that the teacher
// does not list, which a bitmap in LDS leaves out (subtracting the listed ones
// from the whole sum would lose the rest's digits where little is left).
template <typename T>
__global__ __launch_bounds__(kNT) void distill_kernel(DistillArgs a, int64_t row0, int segs, int cps)
{
    constexpr int U = 4, W = Row<T>::W;
    __shared__ Total tot[kNW];
    __shared__ Teacher te;
    __shared__ unsigned bits[kBitWords];
    const int64_t row_i = row0 + blockIdx.x / segs;
    const int seg = blockIdx.x % segs, tid = threadIdx.x, K = a.top_k, lane = tid & (kWave - 1);
    const int32_t *index = a.top_index + row_i * K;
    const float *value = a.top_value + row_i * K;
    const Row<T> row(a.in.logits, row_i * a.in.stride, a.in.vocab);
    const int k0 = min(seg * cps, row.chunks), k1 = min(k0 + cps, row.chunks);
    const int lo = max(k0, row.full_lo), hi = min(k1, row.full_hi);
    if (is_padding(index, value, K, lane)) {
        if (segs == 1)
            pad_distill(a.loss, a.stats, row_i);
        return;
    }
    if (tid < kWave) {
        mark_listed(bits, ((k1 - k0) * W + 31) / 32, index, K, row.phase - k0 * W, (k1 - k0) * W,
                    a.in.vocab, lane);
        if (segs == 1) {
            read_teacher(te, index, value, K, a.mode, a.in.vocab, lane);
            read_listed(te, row.p, (double)a.in.scale, lane);
        }
    }
    __syncthreads();
    const Scale sc(a.in.c);
    Sum q;
    auto take = [&](const Chunk<T> &ch, int k) {
        float x[W];
        ch.widen(x);
        const int at = (k - k0) * W;
        const unsigned listed = bits[at >> 5] >> (at & 31) & ((1u << W) - 1);
        if (listed) {
#pragma unroll
            for (int i = 0; i < W; ++i)
                x[i] = listed >> i & 1 ? -kInf : x[i];
        }
        q.add<W, false>(x, sc);
    };
    int k = lo + tid;
    for (; k + kNT * (U - 1) < hi; k += kNT * U) {
        Chunk<T> ch[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            ch[u].stream(row.chunk(k + kNT * u));
#pragma unroll
        for (int u = 0; u < U; ++u)
            take(ch[u], k + kNT * u);
    }
    for (; k < hi; k += kNT) {
        Chunk<T> ch;
        ch.stream(row.chunk(k));
        take(ch, k);
    }
    const int e = tid < 2 * W ? row.edge(tid, k0, k1) : -1;
    if (e >= 0) {
        const int at = e + row.phase - k0 * W;
        const float x[1] = {bits[at >> 5] >> (at & 31) & 1 ? -kInf : row.at(e)};
        q.add<1, false>(x, sc);
    }
    const Total t = block_total<false>(q, sc, tot);
    if (segs > 1) {
        if (tid == 0)
            a.parts[row_i * segs + seg] = LossPart{t.m, t.s, 0.0f, 0.0f};
    } else if (tid < kWave) {
        finish_distill(te, t, K, a.in, a.loss, a.stats, row_i, lane);
    }
}

template <typename T>
__global__ __launch_bounds__(kNT) void distill_join_kernel(DistillArgs a, int64_t row0, int segs)
{
    __shared__ Total tot[kNW];
    __shared__ Teacher te;
    const int64_t r = row0 + blockIdx.x;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), K = a.top_k;
    const int32_t *index = a.top_index + r * K;
    const float *value = a.top_value + r * K;
    if (is_padding(index, value, K, lane)) {
        pad_distill(a.loss, a.stats, r);
        return;
    }
    if (tid < kWave) {
        read_teacher(te, index, value, K, a.mode, a.in.vocab, lane);
        read_listed(te, static_cast<const T *>(a.in.logits) + r * a.in.stride, (double)a.in.scale, lane);
    }
    const Total t = join_parts(a.parts + r * segs, segs, Scale(a.in.c), tot);
    if (tid < kWave)
        finish_distill(te, t, K, a.in, a.loss, a.stats, r, lane);
}

// d_logits_j = w (Q p_j - q_j) for a listed token and w (Q p_rest - q_rest)
// p_j / p_rest for the others (w = scale d_loss, Q the teacher's total), where
// p_j / p_rest is the softmax over the tokens that are not listed.  Every
// element is written in the second form first, then the listed ones again.
template <typename T>
__global__ __launch_bounds__(kNT) void distill_grad_kernel(DistillGradArgs a, int64_t row0, int segs,
                                                           int cps)
{
    constexpr int W = Row<T>::W;
    __shared__ Teacher te;
    const int64_t r = row0 + blockIdx.x / segs;
    const int seg = blockIdx.x % segs, tid = threadIdx.x, lane = tid & (kWave - 1), K = a.top_k;
    const Row<T> row(a.in.logits, r * a.in.stride, a.in.vocab);
    T *out = static_cast<T *>(a.d_logits) + r * a.d_stride;
    const int k0 = min(seg * cps, row.chunks), k1 = min(k0 + cps, row.chunks);
    const float dl = a.d_loss[r];
    const float m = a.stats[4 * r], ln = a.stats[4 * r + 1];
    const float tm = a.stats[4 * r + 2], tln = a.stats[4 * r + 3];
    const double scale = (double)a.in.scale, w = (double)dl * scale;
    if (tid < kWave) {
        read_teacher(te, a.top_index + r * K, a.top_value + r * K, K, a.mode, a.in.vocab, lane);
        wave_sync();
        read_listed(te, row.p, scale, lane);
    }
    __syncthreads();   // in place: the listed logits are read before any is overwritten
    const bool zero = !te.any || dl == 0.0f;
    if (zero || te.bad || m == -kInf) {
        fill_row(row, out, k0, k1, te.bad && !zero ? __builtin_nanf("") : 0.0f);
        return;
    }
    if (tm == -kInf) {
        fill_row(row, out, k0, k1, 0.0f);
    } else {
        const Scale k(a.in.c);
        const float c = k.c, ref = tm * c;
        const double rest_p = exp(((double)tm - (double)m) * scale + (double)tln - (double)ln);
        const float off = residue(tm, k) + tln * 1.44269504088896340736f;
        const float coef = (float)(w * (te.total * rest_p - te.rest)) * pow2(-off);
        if (__builtin_fabsf(tm) > k.big)
            map_row(row, out, k0, k1, -1, 0.0f, [&](float x) { return coef * pow2((x - tm) * c); });
        else
            map_row(row, out, k0, k1, -1, 0.0f,
                    [&](float x) { return coef * pow2(__builtin_fmaf(x, c, -ref)); });
    }
    __syncthreads();
    // the listed tokens of this segment
    const int id = tid < K ? te.lead[tid] : -1, at = id + row.phase;
    if (id >= 0 && at >= k0 * W && at < k1 * W) {
        store_one(out + id, listed_grad(te, tid, (double)m, (double)ln, w, scale));
    }
}

// -- forward and backward of a row held in registers --------------------------------------
//
// One workgroup of NT threads holds a row of up to 16 chunks a thread in its
// registers: the logits are read from memory once, summed as they arrive, and
// turned into gradients from the registers.

constexpr int kHeld = 16;

template <typename T, int NT>
struct HeldRow {
    static constexpr int W = Row<T>::W;
    Chunk<T> ch[kHeld];
    float edge;   // of the row's partial first and last chunk
    int lo, hi, e;

    __device__ __forceinline__ explicit HeldRow(const Row<T> &row)
        : lo(row.full_lo + (int)threadIdx.x), hi(row.full_hi)
    {
        constexpr unsigned none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;   // -inf
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            ch[i].r = __builtin_bit_cast(decltype(ch[i].r), u32x4{none, none, none, none});
            if (lo + NT * i < hi)
                ch[i].stream(row.chunk(lo + NT * i));
        }
        e = (int)threadIdx.x < 2 * W ? row.edge(threadIdx.x, 0, row.chunks) : -1;
        edge = e >= 0 ? row.at(e) : -kInf;
    }
    // Some thread has an i-th chunk.
    __device__ __forceinline__ bool any(const Row<T> &row, int i) const
    {
        return row.full_lo + NT * i < hi;
    }
    // Writes f(logit) for every element the thread holds; element `hot` gets
    // `add` more.
    template <typename F>
    __device__ __forceinline__ void map(const Row<T> &row, T *out, int hot, float add, F f) const
    {
        const int hot_k = hot < 0 ? -1 : (hot + row.phase) / W, hot_i = (hot + row.phase) & (W - 1);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int k = lo + NT * i;
            if (k < hi) {
                float x[W], g[W];
                ch[i].widen(x);
#pragma unroll
                for (int j = 0; j < W; ++j)
                    g[j] = f(x[j]);
                if (k == hot_k) {
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        g[j] = j == hot_i ? g[j] + add : g[j];
                }
                store_chunk(out + (k * W - row.phase), g);
            }
        }
        if (e >= 0) {
            const float g = f(edge);
            store_one(out + e, e == hot ? g + add : g);
        }
    }
};

template <typename T, int NT, bool ENT>
__global__ __launch_bounds__(NT) void logprob_row_kernel(LogprobArgs a, LogprobGradArgs b, int64_t row0)
{
    constexpr int W = Row<T>::W;
    __shared__ Total tot[NT / kWave];
    const int64_t r = row0 + blockIdx.x;
    const Row<T> row(a.in.logits, r * a.in.stride, a.in.vocab);
    T *out = static_cast<T *>(b.d_logits) + r * b.d_stride;
    const int64_t tok = a.tokens ? a.tokens[r] : 0;
    if (tok < 0) {
        pad_logprob(a, r);
        fill_row<T, NT>(row, out, 0, row.chunks, 0.0f);
        return;
    }
    const float l = token_logit<T>(a, r);   // in place: before it is overwritten
    const HeldRow<T, NT> held(row);
    const float dl = b.d_logprob ? b.d_logprob[r] : 0.0f;
    const float dh = b.d_entropy ? b.d_entropy[r] : 0.0f;
    const Scale k(a.in.c);
    Sum q;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (held.any(row, i)) {
            float x[W];
            held.ch[i].widen(x);
            q.template add<W, ENT>(x, k);
        }
    if (held.e >= 0) {
        const float x[1] = {held.edge};
        q.template add<1, ENT>(x, k);
    }
    const Total t = block_total<ENT, NT / kWave>(q, k, tot);
    finish_logprob(a, r, l, t);
    const bool zero = dl == 0.0f && dh == 0.0f, bad = tok >= a.in.vocab;
    if (zero || bad || t.empty()) {
        fill_row<T, NT>(row, out, 0, row.chunks, bad && !zero ? __builtin_nanf("") : 0.0f);
        return;
    }
    // log2 p = t - log2 S
    const float m = t.m, ref = m * k.c, log2s = log2f(t.s), inv = a.in.scale / t.s;
    const float h = ENT ? kLn2 * (log2s - t.a / t.s) : 0.0f;
    const float u = -inv * (ENT ? dl + dh * (h - kLn2 * log2s) : dl), v = ENT ? -inv * dh * kLn2 : 0.0f;
    const int hot = b.d_logprob ? (int)tok : -1;
    auto grad = [&](float x) { return pow2(x) * (ENT ? __builtin_fmaf(v, __builtin_fmaxf(x, kTiny), u) : u); };
    if (__builtin_fabsf(m) > k.big)
        held.map(row, out, hot, a.in.scale * dl, [&](float x) { return grad((x - m) * k.c); });
    else
        held.map(row, out, hot, a.in.scale * dl,
                 [&](float x) { return grad(__builtin_fmaf(x, k.c, -ref)); });
}

template <typename T, int NT>
__global__ __launch_bounds__(NT) void distill_row_kernel(DistillArgs a, DistillGradArgs b, int64_t row0)
{
    constexpr int W = Row<T>::W;
    constexpr int kWords = (NT * kHeld * W + 2 * W + 31) / 32;
    __shared__ Total tot[NT / kWave];
    __shared__ Teacher te;
    __shared__ unsigned bits[kWords];
    const int64_t r = row0 + blockIdx.x;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), K = a.top_k;
    const Row<T> row(a.in.logits, r * a.in.stride, a.in.vocab);
    T *out = static_cast<T *>(b.d_logits) + r * b.d_stride;
    const int32_t *index = a.top_index + r * K;
    const float *value = a.top_value + r * K;
    if (is_padding(index, value, K, lane)) {
        pad_distill(a.loss, a.stats, r);
        fill_row<T, NT>(row, out, 0, row.chunks, 0.0f);
        return;
    }
    HeldRow<T, NT> held(row);
    const double scale = (double)a.in.scale;
    if (tid < kWave) {
        mark_listed(bits, (row.chunks * W + 31) / 32, index, K, row.phase, row.chunks * W, a.in.vocab,
                    lane);
        read_teacher(te, index, value, K, a.mode, a.in.vocab, lane);
        read_listed(te, row.p, scale, lane);
    }
    __syncthreads();
    const Scale k(a.in.c);
    Sum q;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (held.any(row, i)) {
            const int at = (held.lo + NT * i) * W;
            float x[W];
            held.ch[i].widen(x);
            const unsigned listed = held.lo + NT * i < held.hi
                                        ? bits[at >> 5] >> (at & 31) & ((1u << W) - 1) : 0u;
            if (listed) {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    x[j] = listed >> j & 1 ? -kInf : x[j];
            }
            q.template add<W, false>(x, k);
        }
    if (held.e >= 0) {
        const int at = held.e + row.phase;
        const float x[1] = {bits[at >> 5] >> (at & 31) & 1 ? -kInf : held.edge};
        q.template add<1, false>(x, k);
    }
    const Total t = block_total<false, NT / kWave>(q, k, tot);
    if (tid < kWave)
        finish_distill(te, t, K, a.in, a.loss, a.stats, r, lane);
    const float dl = b.d_loss[r];
    const double w = (double)dl * scale;
    const bool nothing = t.empty() && te.listed_sum == 0.0;
    if (dl == 0.0f || te.bad || nothing) {
        fill_row<T, NT>(row, out, 0, row.chunks, te.bad && dl != 0.0f ? __builtin_nanf("") : 0.0f);
        return;
    }
    // the rest's share of the whole sum, then the coefficient of 2^t
    const float lm = __builtin_fmaxf((float)te.listed_max, kLowest);
    const float share = t.s / (t.s + (float)te.listed_sum * pow2(((double)lm - (double)t.m) * (double)k.c));
    const float coef = t.empty() ? 0.0f : (float)(w * (te.total * (double)share - te.rest)) / t.s;
    const float m = t.m, ref = m * k.c;
    if (t.empty())
        fill_row<T, NT>(row, out, 0, row.chunks, 0.0f);
    else if (__builtin_fabsf(m) > k.big)
        held.map(row, out, -1, 0.0f, [&](float x) { return coef * pow2((x - m) * k.c); });
    else
        held.map(row, out, -1, 0.0f, [&](float x) { return coef * pow2(__builtin_fmaf(x, k.c, -ref)); });
    __syncthreads();
    for (int i = tid; i < K; i += NT)
        if (te.lead[i] >= 0)
            store_one(out + te.lead[i], listed_grad(te, i, te.max, te.ln, w, scale));
}

// -- launches ---------------------------------------------------------------------------------

// Calls f(first row, rows) so that no launch has more than 2^31 threads.
template <typename F>
int each_launch(int64_t rows, int per_row, F f, int threads = kNT)
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

// Chunks per workgroup when a row of `vocab` elements at any 16-byte phase is
// cut for `segs` workgroups.
template <typename T>
int chunks_per(int vocab, int segs)
{
    constexpr int W = 16 / (int)sizeof(T);
    const int most = (vocab + 2 * (W - 1)) / W;
    return (most + segs - 1) / segs;
}

template <typename T, bool ENT, bool TOP>
int launch_logprob_t(const LogprobArgs &a, int segs, hipStream_t st)
{
    const int cps = chunks_per<T>(a.in.vocab, segs);
    if (int e = each_launch(a.in.rows, segs, [&](int64_t r, unsigned n) {
            hipLaunchKernelGGL((logprob_kernel<T, ENT, TOP>), dim3(n * (unsigned)segs), dim3(kNT), 0,
                               st, a, r, segs, cps);
        }))
        return e;
    if (segs == 1)
        return hipSuccess;
    return each_launch(a.in.rows, 1, [&](int64_t r, unsigned n) {
        hipLaunchKernelGGL((logprob_join_kernel<TOP>), dim3(n), dim3(kNT), 0, st, a, r, segs);
    });
}

template <typename T>
int launch_logprob_of(const LogprobArgs &a, int segs, hipStream_t st)
{
    if (a.with_entropy)
        return a.top_k ? launch_logprob_t<T, true, true>(a, segs, st)
                       : launch_logprob_t<T, true, false>(a, segs, st);
    return a.top_k ? launch_logprob_t<T, false, true>(a, segs, st)
                   : launch_logprob_t<T, false, false>(a, segs, st);
}

template <typename T>
int launch_distill_of(const DistillArgs &a, int segs, hipStream_t st)
{
    const int cps = chunks_per<T>(a.in.vocab, segs);
    if (int e = each_launch(a.in.rows, segs, [&](int64_t r, unsigned n) {
            hipLaunchKernelGGL((distill_kernel<T>), dim3(n * (unsigned)segs), dim3(kNT), 0, st, a, r,
                               segs, cps);
        }))
        return e;
    if (segs == 1)
        return hipSuccess;
    return each_launch(a.in.rows, 1, [&](int64_t r, unsigned n) {
        hipLaunchKernelGGL((distill_join_kernel<T>), dim3(n), dim3(kNT), 0, st, a, r, segs);
    });
}

// Threads of the workgroup that holds a row in registers; 0: the row is too
// long for 1024.
template <typename T>
int held_threads(int vocab)
{
    const int most = chunks_per<T>(vocab, 1);
    return most <= 64 * kHeld ? 64 : most <= 256 * kHeld ? 256 : most <= 512 * kHeld ? 512
         : most <= 1024 * kHeld ? 1024 : 0;
}

template <typename T, int NT>
int launch_logprob_row_nt(const LogprobArgs &a, const LogprobGradArgs &b, hipStream_t st)
{
    return each_launch(a.in.rows, 1, [&](int64_t r, unsigned n) {
        if (a.with_entropy)
            hipLaunchKernelGGL((logprob_row_kernel<T, NT, true>), dim3(n), dim3(NT), 0, st, a, b, r);
        else
            hipLaunchKernelGGL((logprob_row_kernel<T, NT, false>), dim3(n), dim3(NT), 0, st, a, b, r);
    }, NT);
}
template <typename T>
int launch_logprob_row(const LogprobArgs &a, const LogprobGradArgs &b, int threads, hipStream_t st)
{
    return threads == 64  ? launch_logprob_row_nt<T, 64>(a, b, st)
         : threads == 256 ? launch_logprob_row_nt<T, 256>(a, b, st)
         : threads == 512 ? launch_logprob_row_nt<T, 512>(a, b, st)
                          : launch_logprob_row_nt<T, 1024>(a, b, st);
}
template <typename T, int NT>
int launch_distill_row_nt(const DistillArgs &a, const DistillGradArgs &b, hipStream_t st)
{
    return each_launch(a.in.rows, 1, [&](int64_t r, unsigned n) {
        hipLaunchKernelGGL((distill_row_kernel<T, NT>), dim3(n), dim3(NT), 0, st, a, b, r);
    }, NT);
}
template <typename T>
int launch_distill_row(const DistillArgs &a, const DistillGradArgs &b, int threads, hipStream_t st)
{
    return threads == 64  ? launch_distill_row_nt<T, 64>(a, b, st)
         : threads == 256 ? launch_distill_row_nt<T, 256>(a, b, st)
         : threads == 512 ? launch_distill_row_nt<T, 512>(a, b, st)
                          : launch_distill_row_nt<T, 1024>(a, b, st);
}

// Workgroups per row of a gradient pass: 8 chunks per thread.
template <typename T>
int grad_segments(int vocab)
{
    constexpr int W = 16 / (int)sizeof(T);
    return (vocab + 8 * kNT * W - 1) / (8 * kNT * W);
}

}  // namespace

int launch_logprob(const LogprobArgs &a, int32_t segs, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return a.in.dtype == ZERO_BF16 ? launch_logprob_of<uint16_t>(a, segs, st)
                                   : launch_logprob_of<float>(a, segs, st);
}

bool loss_row_held(const LossRows &in)
{
    return (in.dtype == ZERO_BF16 ? held_threads<uint16_t>(in.vocab) : held_threads<float>(in.vocab)) > 0;
}

int launch_logprob_fused(const LogprobArgs &a, const LogprobGradArgs &b, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return a.in.dtype == ZERO_BF16
               ? launch_logprob_row<uint16_t>(a, b, held_threads<uint16_t>(a.in.vocab), st)
               : launch_logprob_row<float>(a, b, held_threads<float>(a.in.vocab), st);
}

int launch_distill_fused(const DistillArgs &a, const DistillGradArgs &b, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return a.in.dtype == ZERO_BF16
               ? launch_distill_row<uint16_t>(a, b, held_threads<uint16_t>(a.in.vocab), st)
               : launch_distill_row<float>(a, b, held_threads<float>(a.in.vocab), st);
}

int launch_logprob_grad(const LogprobGradArgs &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const bool bf = a.in.dtype == ZERO_BF16, ent = a.d_entropy != nullptr;
    const int segs = bf ? grad_segments<uint16_t>(a.in.vocab) : grad_segments<float>(a.in.vocab);
    const int cps = bf ? chunks_per<uint16_t>(a.in.vocab, segs) : chunks_per<float>(a.in.vocab, segs);
    return each_launch(a.in.rows, segs, [&](int64_t r, unsigned n) {
        const dim3 grid(n * (unsigned)segs), block(kNT);
        if (bf && ent)
            hipLaunchKernelGGL((logprob_grad_kernel<uint16_t, true>), grid, block, 0, st, a, r, segs, cps);
        else if (bf)
            hipLaunchKernelGGL((logprob_grad_kernel<uint16_t, false>), grid, block, 0, st, a, r, segs, cps);
        else if (ent)
            hipLaunchKernelGGL((logprob_grad_kernel<float, true>), grid, block, 0, st, a, r, segs, cps);
        else
            hipLaunchKernelGGL((logprob_grad_kernel<float, false>), grid, block, 0, st, a, r, segs, cps);
    });
}

int launch_distill(const DistillArgs &a, int32_t segs, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return a.in.dtype == ZERO_BF16 ? launch_distill_of<uint16_t>(a, segs, st)
                                   : launch_distill_of<float>(a, segs, st);
}

int launch_distill_grad(const DistillGradArgs &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const bool bf = a.in.dtype == ZERO_BF16;
    const int segs = bf ? grad_segments<uint16_t>(a.in.vocab) : grad_segments<float>(a.in.vocab);
    const int cps = bf ? chunks_per<uint16_t>(a.in.vocab, segs) : chunks_per<float>(a.in.vocab, segs);
    return each_launch(a.in.rows, segs, [&](int64_t r, unsigned n) {
        const dim3 grid(n * (unsigned)segs), block(kNT);
        if (bf)
            hipLaunchKernelGGL((distill_grad_kernel<uint16_t>), grid, block, 0, st, a, r, segs, cps);
        else
            hipLaunchKernelGGL((distill_grad_kernel<float>), grid, block, 0, st, a, r, segs, cps);
    });
}

}  // namespace zero
