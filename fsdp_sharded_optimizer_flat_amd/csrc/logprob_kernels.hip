// logprob_kernels.hip -- log probabilities of given tokens, with entropy and the
// top alternatives, over rows of logits, forward and backward.
#include <type_traits>

#include "token_loss_device.h"

namespace zero {
namespace {

using namespace dev;

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
    const T *p = static_cast<const T *>(a.in.logits) + row_i * a.in.stride;
    const Row<T> row(p, a.in.vocab);
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

// d_logits_j = scale (d_lp ([j = t] - p_j) - d_H p_j (ln p_j + H)).  With p_j =
// 2^t inv this is [j = t] scale d_lp - p_j (u + v t), u and v the row's.
// One workgroup per kNT chunks of a row, one to a thread: neighbouring workgroups
// sweep the memory in order, as a copy does.
template <typename T, bool ENT>
__global__ __launch_bounds__(kNT) void logprob_grad_kernel(LogprobGradArgs a, int64_t row0, int segs)
{
    const int64_t r = row0 + blockIdx.x / segs;
    const int k0 = (int)(blockIdx.x % segs) * kNT;
    T *out = static_cast<T *>(a.d_logits) + r * a.d_stride;
    const Row<T> row(static_cast<const T *>(a.in.logits) + r * a.in.stride, a.in.vocab);
    const RowPart<T, kNT, 1> seg(row, k0);   // on its way while the row's values are read
    const int64_t tok = a.tokens ? ld_uniform(a.tokens + r) : 0;
    const float dl = a.d_logprob ? ld_uniform(a.d_logprob + r) : 0.0f;
    const float dh = ENT ? ld_uniform(a.d_entropy + r) : 0.0f;
    const float m = ld_uniform(a.stats + 2 * r), ln = ld_uniform(a.stats + 2 * r + 1);
    const bool zero = tok < 0 || (dl == 0.0f && dh == 0.0f), bad = tok >= a.in.vocab;
    if (zero || bad || m == -kInf) {
        fill_row(row, out, k0, k0 + kNT, bad && !zero ? __builtin_nanf("") : 0.0f);
        return;
    }
    const Scale k(a.in.c);
    // log2 p = t - off
    const float ref = m * k.c, off = residue(m, k) + ln * kLog2E;
    const float inv = pow2(-off);
    const float h = ENT ? ld_uniform(a.entropy + r) : 0.0f;
    const float u = -a.in.scale * (dl + dh * (h - off * kLn2)) * inv;
    const float v = -a.in.scale * dh * kLn2 * inv;
    // the given token's thread; in place: it reads the logit before it writes
    const bool mine = a.d_logprob && owner_of<T, kNT>(row, (int)tok, k0, kNT) == (int)threadIdx.x;
    const float l = mine ? row.at((int)tok) : 0.0f;
    auto grad = [&](float t) { return pow2(t) * (ENT ? __builtin_fmaf(v, __builtin_fmaxf(t, kTiny), u) : u); };
    if (__builtin_fabsf(m) > k.big)
        seg.map(row, out, [&](float x) { return grad((x - m) * k.c); });
    else
        seg.map(row, out, [&](float x) { return grad(__builtin_fmaf(x, k.c, -ref)); });
    // after the same thread's own store of the element
    if (mine)
        store_one(out + tok, grad(rel(l, m, ref, k)) + a.in.scale * dl);
}

constexpr int kHeld = 16;   // chunks a thread holds

// Forward and backward of whole rows, at most kHeld NT chunks each.
template <typename T, int NT, bool ENT, bool SAME>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(4)))
void logprob_row_kernel(LogprobArgs a, LogprobGradArgs b)
{
    typedef HeldRow<T, NT, kHeld, SAME> Held;
    constexpr int N = Held::G * Row<T>::W;
    __shared__ Total tot[2][NT / kWave];
    auto out_at = [&](int64_t r) { return static_cast<T *>(b.d_logits) + r * b.d_stride; };
    auto row_at = [&](int64_t r) {
        return Row<T>(static_cast<const T *>(a.in.logits) + r * a.in.stride, a.in.vocab);
    };
    // The next row from r on that is not padding (padding rows are finished on
    // the way), or a.in.rows.
    auto skip_padding = [&](int64_t r) {
        while (r < a.in.rows && a.tokens && ld_uniform(a.tokens + r) < 0) {
            const Row<T> row = row_at(r);
            pad_logprob(a, r);
            fill_row<T, NT>(row, out_at(r), 0, row.chunks, 0.0f);
            r += gridDim.x;
        }
        return r;
    };
    const Scale k(a.in.c);
    __shared__ u32x4 park[NT * parked(NT) + 1];
    Held held;
    held.park = park;
    int64_t r = skip_padding(blockIdx.x);
    if (r >= a.in.rows)
        return;
    held.read(row_at(r));
    held.take(row_at(r));
    for (int turn = 0;; turn ^= 1) {
        const int64_t rn = skip_padding(r + gridDim.x);
        const Row<T> next = rn < a.in.rows ? row_at(rn) : Row<T>();
        const float l = token_logit<T>(a, r);   // in place: before it is overwritten
        const int64_t tok = a.tokens ? ld_uniform(a.tokens + r) : 0;
        const float dl = b.d_logprob ? ld_uniform(b.d_logprob + r) : 0.0f;
        const float dh = b.d_entropy ? ld_uniform(b.d_entropy + r) : 0.0f;
        Sum q;
        held.each_group([&](int, const float (&x)[N]) { q.template add<N, ENT>(x, k); });
        if (held.e >= 0) {
            const float x[1] = {held.edge};
            q.template add<1, ENT>(x, k);
        }
        // two sets of LDS slots: a wave may still read this row's when another
        // writes the next row's
        const Total t = block_total<ENT, NT / kWave>(q, k, tot[turn]);
        finish_logprob(a, r, l, t);
        T *out = out_at(r);
        const bool zero = dl == 0.0f && dh == 0.0f, bad = tok >= a.in.vocab;
        const bool fill = zero || bad || t.empty(), big = __builtin_fabsf(t.m) > k.big;
        // log2 p = t - log2 S
        const float m = t.m, ref = m * k.c, log2s = log2f(t.s), inv = a.in.scale / t.s;
        const float h = ENT ? kLn2 * (log2s - t.a / t.s) : 0.0f;
        const float u = -inv * (ENT ? dl + dh * (h - kLn2 * log2s) : dl);
        const float v = ENT ? -inv * dh * kLn2 : 0.0f;
        auto grad = [&](float x) {
            return pow2(x) * (ENT ? __builtin_fmaf(v, __builtin_fmaxf(x, kTiny), u) : u);
        };
        if (fill)
            fill_row<T, NT>(held.row, out, 0, held.row.chunks, bad && !zero ? __builtin_nanf("") : 0.0f);
        else if (big) {   // rare: from memory, so that the held row's code is not there twice
            for (int k0 = 0; k0 < held.row.chunks; k0 += NT)
                RowPart<T, NT, 1>(held.row, k0).map(held.row, out, [&](float x) { return grad((x - m) * k.c); });
            __syncthreads();
        }
        held.map(out, !fill && !big, next, [&](float x) { return grad(__builtin_fmaf(x, k.c, -ref)); });
        // the given token's, after its thread's own store of the element
        const int owner = owner_of<T, NT>(held.row, (int)tok, 0, held.row.chunks);
        if (b.d_logprob && !fill && (int)threadIdx.x == (big ? 0 : owner))
            store_one(out + tok, grad(rel(l, m, ref, k)) + a.in.scale * dl);
        held.take(next);
        if (rn >= a.in.rows)
            return;
        r = rn;
    }
}

// -- launches ---------------------------------------------------------------------------------

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
    const dim3 grid(held_grid(a.in.rows, NT));
    const bool same = same_phase(a.in, b.d_logits, b.d_stride);
    if (a.with_entropy && same)
        hipLaunchKernelGGL((logprob_row_kernel<T, NT, true, true>), grid, dim3(NT), 0, st, a, b);
    else if (a.with_entropy)
        hipLaunchKernelGGL((logprob_row_kernel<T, NT, true, false>), grid, dim3(NT), 0, st, a, b);
    else if (same)
        hipLaunchKernelGGL((logprob_row_kernel<T, NT, false, true>), grid, dim3(NT), 0, st, a, b);
    else
        hipLaunchKernelGGL((logprob_row_kernel<T, NT, false, false>), grid, dim3(NT), 0, st, a, b);
    return hipGetLastError();
}
template <typename T>
int launch_logprob_row(const LogprobArgs &a, const LogprobGradArgs &b, hipStream_t st)
{
    const int threads = held_threads<T>(a.in.vocab);
    return threads == 64  ? launch_logprob_row_nt<T, 64>(a, b, st)
         : threads == 256 ? launch_logprob_row_nt<T, 256>(a, b, st)
         : threads == 512 ? launch_logprob_row_nt<T, 512>(a, b, st)
                          : launch_logprob_row_nt<T, 1024>(a, b, st);
}

}  // namespace

int launch_logprob(const LogprobArgs &a, int32_t segs, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return a.in.dtype == ZERO_BF16 ? launch_logprob_of<uint16_t>(a, segs, st)
                                   : launch_logprob_of<float>(a, segs, st);
}

int launch_logprob_grad(const LogprobGradArgs &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    const bool bf = a.in.dtype == ZERO_BF16, ent = a.d_entropy != nullptr;
    const int segs = ((bf ? chunks_per<uint16_t>(a.in.vocab, 1) : chunks_per<float>(a.in.vocab, 1)) + kNT - 1) / kNT;
    return each_launch(a.in.rows, segs, [&](int64_t r, unsigned n) {
        const dim3 grid(n * (unsigned)segs), block(kNT);
        if (bf && ent)
            hipLaunchKernelGGL((logprob_grad_kernel<uint16_t, true>), grid, block, 0, st, a, r, segs);
        else if (bf)
            hipLaunchKernelGGL((logprob_grad_kernel<uint16_t, false>), grid, block, 0, st, a, r, segs);
        else if (ent)
            hipLaunchKernelGGL((logprob_grad_kernel<float, true>), grid, block, 0, st, a, r, segs);
        else
            hipLaunchKernelGGL((logprob_grad_kernel<float, false>), grid, block, 0, st, a, r, segs);
    });
}

bool logprob_row_held(const LossRows &in)
{
    return (in.dtype == ZERO_BF16 ? held_threads<uint16_t>(in.vocab) : held_threads<float>(in.vocab)) > 0;
}

int launch_logprob_fused(const LogprobArgs &a, const LogprobGradArgs &b, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    return a.in.dtype == ZERO_BF16 ? launch_logprob_row<uint16_t>(a, b, st)
                                   : launch_logprob_row<float>(a, b, st);
}

}  // namespace zero
