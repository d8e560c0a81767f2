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
// leaves the largest logit of each group of kGroup in LDS (its upper 16 bits); a
// group is a whole cache line of bf16, so that reading it again costs no more.  Of
// its groups each wave finds the ceil(K / waves)-th largest maximum by bisection;
// the least of these is a bound that at least K logits reach.  Only groups that
// reach it are read again (a little more than K of them), and their logits that
// reach it become candidates, each ranked by the number of larger ones.  Where
// there are too many (plateaus of equal logits, few groups), a radix search over
// the whole keys, which are all different, finds the K-th exactly.

constexpr int kIndexBits = 20;
static_assert(ZERO_MAX_VOCAB <= 1 << kIndexBits, "the index fits its field");
constexpr int kGroup = 64;
constexpr int kGroups = 2304;   // those of kLossMaxSegment elements, and some to spare
static_assert(kGroups >= (int)(kLossMaxSegment / kGroup) + 2, "a segment's groups fit");

// Binary logarithm of the lanes whose chunks of W elements are a group: kGroup
// elements, or fewer where that leaves less than two groups to an alternative,
// which makes a low bound and many candidates (1500 rows of 15576 bf16, 200
// alternatives: 120 us with groups of kGroup, 35 with smaller ones; 64 of 4000:
// 40 and 12).
template <int W>
constexpr int kGroupLog = W == 4 ? 4 : 3;
template <int W>
__device__ __forceinline__ int group_lanes(int chunks, int K)
{
    static_assert(W << kGroupLog<W> == kGroup && 4 * ZERO_MAX_TOP + 2 <= kGroups, "groups fit");
    int lg = kGroupLog<W>;
    while (lg > 0 && chunks >> lg < 2 * K)
        --lg;
    return lg;
}
// The maximum over 2^lg neighbouring lanes (aligned), in each of them.
template <int W>
__device__ __forceinline__ float group_max(float x, int lg)
{
    if (lg == kGroupLog<W>) {   // one branch in the loop over long rows
        x = __builtin_fmaxf(x, from_lane<kLaneXor1>(x, x));
        x = __builtin_fmaxf(x, from_lane<kLaneXor2>(x, x));
        x = __builtin_fmaxf(x, from_lane<kMirror8>(x, x));
        return W == 4 ? __builtin_fmaxf(x, from_lane<kMirror16>(x, x)) : x;
    }
    if (lg > 0)
        x = __builtin_fmaxf(x, from_lane<kLaneXor1>(x, x));
    if (lg > 1)
        x = __builtin_fmaxf(x, from_lane<kLaneXor2>(x, x));
    if (lg > 2)
        x = __builtin_fmaxf(x, from_lane<kMirror8>(x, x));
    return x;
}
constexpr int kCands = 1024, kPad = 16;

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
    unsigned floor[16];    // each wave's bound
    unsigned long long floor64;
    alignas(16) uint16_t gmax[kGroups];
    uint16_t list[kGroups];
    alignas(16) uint64_t cand[kCands + kPad];
    // the K largest of many candidates, once the groups are done with
    __device__ __forceinline__ uint64_t *best() { return reinterpret_cast<uint64_t *>(gmax); }
};
static_assert((ZERO_MAX_TOP + kPad) * sizeof(uint64_t) <= sizeof(Select::gmax), "room for the best");

// One radix pass's choice: the bin of sh.hist (256 bins) that holds the want-th
// largest entry, and how many lie above it.  Thread b < 256 owns bin b.
__device__ __forceinline__ void pick_bin(Select &sh, unsigned want)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    __syncthreads();
    if (wave < 4) {
        const unsigned own = sh.hist[tid];
        unsigned above = 0;                     // entries in bins above this one
        for (int w = wave + 1; w < 4; ++w)
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

// The K-th largest of the keys that `each` visits (at least K of them, all
// different but for zeros).  each(f) calls f(key) once for every key, over the
// whole workgroup.
template <typename Each>
__device__ uint64_t kth_key(Select &sh, int K, Each each)
{
    uint64_t prefix = 0;
    unsigned want = (unsigned)K;
    for (int sft = 48; sft >= 0; sft -= 8) {   // 32 + 20 bits in seven bytes
        if (threadIdx.x < 256)
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
template <typename T, int NT, typename F>
__device__ __forceinline__ void each_element(const Row<T> &row, int k0, int k1, F f)
{
    constexpr int W = Row<T>::W;
    const int lo = max(k0, row.full_lo), hi = min(k1, row.full_hi);
    for (int k = lo + (int)threadIdx.x; k < hi; k += NT) {
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

// Writes the K largest of the workgroup's n candidates, best first, through
// put(rank, key).  A candidate's rank is the number of larger ones; where there
// are many, a radix search leaves the K largest first.
template <int NT, typename Put>
__device__ __forceinline__ void put_ranked(Select &sh, int n, int K, Put put)
{
    const int tid = threadIdx.x;
    uint64_t *cand = sh.cand;
    if (n > 256 && n > K) {
        const uint64_t kth = kth_key(sh, K, [&](auto f) {
            for (int i = tid; i < n; i += NT)
                f(sh.cand[i]);
        });
        if (tid == 0)
            sh.count = 0;
        __syncthreads();
        cand = sh.best();
        for (int i = tid; i < n; i += NT)
            if (sh.cand[i] >= kth)
                cand[atomicAdd(&sh.count, 1u)] = sh.cand[i];
        n = K;
    }
    if (tid < kPad)   // below every key: they are compared in batches
        cand[n + tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += NT) {
        const uint64_t own = cand[i];
        int rank = 0;
        for (int j = 0; j < n; j += kPad) {   // kPad / 2 reads on their way at once
            ulonglong2 o[kPad / 2];
#pragma unroll
            for (int u = 0; u < kPad / 2; ++u)
                o[u] = *reinterpret_cast<const ulonglong2 *>(cand + j + 2 * u);
#pragma unroll
            for (int u = 0; u < kPad / 2; ++u)
                rank += (o[u].x > own) + (o[u].y > own);
        }
        if (rank < K)
            put(rank, own);
    }
}

// A bound (the upper 16 bits of a logit's order) that at least K logits of the
// groups reach, and the list of the groups that reach it; at most Q to a thread.
template <int NT, int Q>
__device__ __forceinline__ unsigned list_groups(Select &sh, int groups, int K)
{
    constexpr int NW = NT / kWave;
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    unsigned g[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i)
        g[i] = tid + NT * i < groups ? sh.gmax[tid + NT * i] : 0u;
    // the waves with a group for each lane (the first, if none has)
    const int waves = max(min(groups / kWave, NW), 1), want = (K + waves - 1) / waves;
    unsigned bound = 0;
    for (int bit = 15; bit >= 0; --bit) {
        const unsigned v = bound | 1u << bit;
        int have = 0;
#pragma unroll
        for (int i = 0; i < Q; ++i)
            have += __popcll(__ballot(g[i] >= v));
        if (have >= want)
            bound = v;
    }
    if (lane == 0)
        sh.floor[tid / kWave] = tid / kWave < waves ? bound : ~0u;
    if (tid == 0) {
        sh.count = 0;
        sh.listed = 0;
    }
    __syncthreads();
    bound = ~0u;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        bound = min(bound, sh.floor[w]);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < Q; ++i)
        mine += __popcll(__ballot(tid + NT * i < groups && g[i] >= bound));
    unsigned at = 0;
    if (lane == 0 && mine)
        at = atomicAdd(&sh.listed, (unsigned)mine);
    at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const bool in = tid + NT * i < groups && g[i] >= bound;
        const uint64_t m = __ballot(in);
        if (in)
            sh.list[at + __popcll(m & ((uint64_t(1) << lane) - 1))] = (uint16_t)(tid + NT * i);
        at += __popcll(m);
    }
    __syncthreads();
    return bound;
}

// The K largest logits of chunks [k0, k1).  Group g of their whole chunks is places
// g 2^lg .. + 2^lg - 1 of the sweep; sh.gmax holds the upper 16 bits of its largest
// logit's order.
template <typename T, int NT, typename Put>
__device__ void select_top(Select &sh, const Row<T> &row, const Sweep<T> &sweep, int k0, int k1, int lg, int K, Put put)
{
    constexpr int W = Row<T>::W;
    const int tid = threadIdx.x;
    const int lo = sweep.lo, hi = sweep.hi, groups = (sweep.n + (1 << lg) - 1) >> lg;
    const int first = max(k0 * W - row.phase, 0), last = min(k1 * W - row.phase, row.vocab);
    const int n = max(last - first, 0);
    constexpr int Q = (kGroups + NT - 1) / NT, Few = Q < 3 ? Q : 3;
    const unsigned bound = groups <= NT         ? list_groups<NT, 1>(sh, groups, K)
                           : groups <= Few * NT ? list_groups<NT, Few>(sh, groups, K)
                                                : list_groups<NT, Q>(sh, groups, K);
    const float least = bound <= 0x7fu ? -kInf : ord32_value(bound << 16);
    const int todo = (int)sh.listed << lg;
    auto chunk_of = [&](int j) { return sweep.from + (sh.list[j >> lg] << lg) + (j & ((1 << lg) - 1)); };
    auto look = [&](const Chunk<T> &ch, int k) {
        float x[W];
        ch.widen(x);
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (x[i] >= least)
                push(sh, key_of(x[i], k * W - row.phase + i));
    };
    for (int j = tid; j < todo; j += 2 * NT) {   // two reads on their way at once
        const int ka = chunk_of(j), kb = j + NT < todo ? chunk_of(j + NT) : hi;
        Chunk<T> ca, cb;
        const bool has_a = ka >= lo && ka < hi;
        if (has_a)
            ca.load(row.chunk(ka));
        const bool has_b = kb >= lo && kb < hi;
        if (has_b)
            cb.load(row.chunk(kb));
        if (has_a)
            look(ca, ka);
        if (has_b)
            look(cb, kb);
    }
    const int e = tid < 2 * W ? row.edge(tid, k0, k1) : -1;
    if (e >= 0) {
        const float x = row.at(e);
        if (x >= least)
            push(sh, key_of(x, e));
    }
    __syncthreads();
    int cands = (int)sh.count;
    if (cands > kCands) {
        __syncthreads();
        uint64_t kth = 0;
        if (n > K)
            kth = kth_key(sh, K, [&](auto f) {
                each_element<T, NT>(row, k0, k1, [&](float x, int i) { f(key_of(x, i)); });
            });
        if (tid == 0)
            sh.count = 0;
        __syncthreads();
        each_element<T, NT>(row, k0, k1, [&](float x, int i) {
            const uint64_t key = key_of(x, i);
            if (key >= kth)
                push(sh, key);
        });
        __syncthreads();
        cands = min((int)sh.count, kCands);
    }
    put_ranked<NT>(sh, cands, K, put);
}

// -- log probabilities: forward ----------------------------------------------------------

// A row's outputs from its total and the given token's logit (anything where
// the token is outside the vocabulary), by one lane of the workgroup's last wave:
// the first ranks the top alternatives.
__device__ __forceinline__ void finish_logprob(const LogprobArgs &a, int64_t row, float l, const Total &t)
{
    if (threadIdx.x != blockDim.x - kWave)
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
    const int64_t tok = a.tokens ? ld_uniform(a.tokens + row) : -1;
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
    for (int i = from + (int)threadIdx.x; i < a.top_k; i += blockDim.x) {
        a.top_index[row * a.top_k + i] = -1;
        a.top_logprob[row * a.top_k + i] = t.s != t.s ? __builtin_nanf("") : -kInf;
    }
}

// One workgroup per segment of a row (segs of them): the whole result where
// segs is 1, else its LossPart and its top keys.  One pass, U chunks to a thread on
// their way at once, 8 waves on a SIMD: 4096 x 128256 bf16 with entropy 162 us,
// 6.5 TB/s; 2048 x 128256 with the 64 largest of each row 98 us (82 us without: the
// selection is a chain of barriers that other workgroups fill only in part); 64 x
// 128256 with twenty, cut for 1024 workgroups, 18 us with the joining launch,
// both latency: loads, four barriers and a second read of the chosen groups; 1 x
// 50304 with five 10.9 us, one workgroup, half of it for the sums.
template <typename T, int NT, bool ENT, bool TOP>
__global__ __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(NT == kNT ? 8 : 4)))
void logprob_kernel(LogprobArgs a, int64_t row0, int segs, int cps)
{
    constexpr int U = NT == kWide ? 8 : 4, W = Row<T>::W;   // chunks on their way to a thread
    __shared__ Total tot[NT / kWave];
    __shared__ typename std::conditional<TOP, Select, int>::type sh;
    const int64_t row_i = row0 + blockIdx.x / segs;
    const int seg = blockIdx.x % segs, tid = threadIdx.x;
    if (a.tokens && ld_uniform(a.tokens + row_i) < 0) {
        if (segs == 1)
            pad_logprob(a, row_i);
        return;
    }
    const T *p = static_cast<const T *>(a.in.logits) + row_i * a.in.stride;
    const Row<T> row(p, a.in.vocab);
    const int k0 = min(seg * cps, row.chunks), k1 = min(k0 + cps, row.chunks);
    const Sweep<T> sweep(row, k0, k1);
    const float given = segs == 1 ? token_logit<T>(a, row_i) : 0.0f;
    const Scale sc(a.in.c);
    Sum q;
    const int n = sweep.n, lg = group_lanes<W>(n, a.top_k);
    for (int b = 0; b < n; b += NT * U) {
        Chunk<T> ch[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            ch[u] = sweep.read(b + NT * u);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int first = b + NT * u;
            if (first >= n)
                break;
            sweep.trim(ch[u], first, NT);
            float x[W];
            ch[u].widen(x);
            float m = x[0];
#pragma unroll
            for (int i = 1; i < W; ++i)
                m = __builtin_fmaxf(m, x[i]);
            q.add_with_max<W, ENT>(x, m, sc);
            if constexpr (TOP) {
                m = group_max<W>(m, lg);
                if ((tid & ((1 << lg) - 1)) == 0 && first + tid < n)
                    sh.gmax[(first + tid) >> lg] = (uint16_t)(ord32(m) >> 16);
            }
        }
    }
    const int e = tid < 2 * W ? row.edge(tid, k0, k1) : -1;
    if (e >= 0) {
        const float x[1] = {row.at(e)};
        q.add<1, ENT>(x, sc);
    }
    const Total t = block_total<ENT, NT / kWave>(q, sc, tot);
    if (segs > 1 && tid == 0)
        a.parts[row_i * segs + seg] = LossPart{t.m, t.s, t.a, 0.0f};
    if constexpr (TOP) {
        const int elems = max(min(k1 * W - row.phase, row.vocab) - max(k0 * W - row.phase, 0), 0);
        __syncthreads();
        if (t.s != t.s) {   // a NaN or +inf logit: no order, no alternatives
            if (segs == 1)
                put_none(a, row_i, 0, t);
        } else if (segs == 1) {
            const float log2s = log2f(t.s);
            select_top<T, NT>(sh, row, sweep, k0, k1, lg, a.top_k,
                              [&](int r, uint64_t key) { put_top(a, row_i, r, key, t, log2s); });
            put_none(a, row_i, elems, t);
        } else {
            uint64_t *out = a.keys + (row_i * segs + seg) * a.top_k;
            select_top<T, NT>(sh, row, sweep, k0, k1, lg, a.top_k,
                              [&](int r, uint64_t key) { out[r] = key; });
            for (int i = elems + tid; i < a.top_k; i += NT)
                out[i] = 0;   // below every logit's key
        }
    }
    if (segs == 1)
        finish_logprob(a, row_i, given, t);
}

template <bool TOP>
__global__ __launch_bounds__(kNT) void logprob_join_kernel(LogprobArgs a, int64_t row0, int segs)
{
    __shared__ Total tot[kNW];
    __shared__ typename std::conditional<TOP, Select, int>::type sh;
    const int64_t row = row0 + blockIdx.x;
    const int tid = threadIdx.x;
    if (a.tokens && ld_uniform(a.tokens + row) < 0) {
        pad_logprob(a, row);
        return;
    }
    const float given = a.in.dtype == ZERO_BF16 ? token_logit<uint16_t>(a, row) : token_logit<float>(a, row);
    // each segment's alternatives are in order: the least of their ceil(K /
    // segs)-th ones is reached by K
    const int step = (a.top_k + segs - 1) / segs - 1;
    const uint64_t *keys = a.keys + row * segs * a.top_k;
    uint64_t mine = 0, floor = ~uint64_t(0);   // on their way while the parts are added
    if constexpr (TOP) {
        if (tid < segs * a.top_k)
            mine = keys[tid];
        if (tid < segs)
            floor = keys[tid * a.top_k + step];
        if (tid == 0) {
            sh.count = 0;
            sh.floor64 = ~uint64_t(0);
        }
    }
    const Total t = join_parts(a.parts + row * segs, segs, Scale(a.in.c), tot);
    finish_logprob(a, row, given, t);
    if constexpr (TOP) {
        if (t.s != t.s) {
            put_none(a, row, 0, t);
            return;
        }
        const int n = segs * a.top_k;
        const float log2s = log2f(t.s);
        for (int i = tid + kNT; i < segs; i += kNT)
            floor = min(floor, keys[(int64_t)i * a.top_k + step]);
        if (tid < segs)
            atomicMin(&sh.floor64, (unsigned long long)floor);
        __syncthreads();
        uint64_t least = sh.floor64;
        if (least == 0)
            least = 1;   // absent alternatives are zero keys
        for (int i = tid; i < n; i += kNT) {
            const uint64_t key = i == tid ? mine : keys[i];
            if (key >= least)
                push(sh, key);
        }
        __syncthreads();
        if (sh.count > (unsigned)kCands) {
            __syncthreads();
            least = kth_key(sh, a.top_k, [&](auto f) {
                for (int i = tid; i < n; i += kNT)
                    f(keys[i]);
            });
            if (tid == 0)
                sh.count = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kNT)
                if (keys[i] >= max(least, uint64_t(1)))
                    push(sh, keys[i]);
            __syncthreads();
        }
        const int cands = min((int)sh.count, kCands);
        put_ranked<kNT>(sh, cands, a.top_k,
                        [&](int r, uint64_t key) { put_top(a, row, r, key, t, log2s); });
        put_none(a, row, cands, t);
    }
}

// d_logits_j = scale (d_lp ([j = t] - p_j) - d_H p_j (ln p_j + H)).  With p_j =
// 2^t inv this is [j = t] scale d_lp - p_j (u + v t), u and v the row's.
// One workgroup per kNT chunks of a row, one to a thread: neighbouring workgroups
// sweep the memory in order, as a copy does (2048 x 50304 fp32 with an entropy
// gradient: 124 us, 6.6 TB/s; cut for fewer workgroups, several chunks to a thread,
// 159 us; 2048 x 128256 bf16, with or without it: 165 us, 6.4 TB/s).
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
    const bool mine = a.d_logprob && owner_of<T, kNT>(row, (int)tok, k0, kNT, seg.lo) == (int)threadIdx.x;
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

constexpr int kHeld = 16;   // chunks a thread holds: half of its 128 registers

// Forward and backward of whole rows, at most kHeld NT chunks each, read once: 8192
// x 128256 bf16 746 us, 5.6 TB/s (in two launches, each logit read twice, 1175 us);
// 1024 x 50304 42 us; 777 x 50257 fp32 at another phase than its gradient 70 us, at
// the same 65.  A copy kernel of the same loads, barrier and stores, without the
// mathematics, takes 712 us for 8192 rows of 256512 bytes, 39 for 1024 of 100608 and 62
// for 777 of 201024.  1024 threads of 64 registers, half the row to each, spill: 64
// us for 1024 x 50304.
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
        const int owner = owner_of<T, NT>(held.row, (int)tok, 0, held.row.chunks, 0);
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
    if (segs == 1 && wide_rows(a.in)) {
        hipLaunchKernelGGL((logprob_kernel<T, kWide, ENT, TOP>), dim3((unsigned)a.in.rows), dim3(kWide), 0,
                           st, a, (int64_t)0, 1, cps);
        return hipGetLastError();
    }
    if (int e = each_launch(a.in.rows, segs, [&](int64_t r, unsigned n) {
            hipLaunchKernelGGL((logprob_kernel<T, kNT, ENT, TOP>), dim3(n * (unsigned)segs), dim3(kNT), 0,
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
