// sequence_loss_kernels.hip -- losses over packed sequences of tokens' log
// probabilities: the clipped policy loss with a KL term and the preference loss
// over pairs, with their gradients.
//
// All terms are binary64: a difference of two binary32 log probabilities is exact
// there, so whether a ratio is beyond the clipping border is decided on
// logprob - old against the border's logarithm, exp(x) - 1 - x (about x^2 / 2, x often
// 10^-3) keeps its digits, and sums over long sequences lose nothing.  MI355X adds and
// multiplies binary64 as fast as unpacked binary32.
//
// Short calls are bound by their way to the device: 1 sequence of 1024 positions is 3.6
// us of kernel and 8.2 us from call to call.  Long ones by a wave's chain of search, loads,
// terms and sums: 300 sequences of 3400 with a KL term take 10.4 us for the terms, two
// exponentials a target in some 90 binary64 instructions, and 5.6 to scale the
// gradients, where the memory's traffic is 4.3 us; 128 pairs of sequences of 4000, a
// subtraction a target, 4.7 and 7.1 of 3.1.
//
// Few positions: a workgroup to a sequence or pair, one launch.  Many: the array is
// cut into tiles and a wave takes what a sequence has of one, so the work is even
// whatever the lengths.  Share (b, tile) has slot tile + b: the tiles of the sequences
// before b end at or before the one b begins in, so no two shares meet in a slot, and
// the slot's b is found by search.  A second launch adds up each sequence's shares, in
// order, and scales the gradients.
#include <algorithm>

#include "device_common.h"
#include "sequence_loss.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kQuadTokens = 4;   // positions of a lane
static_assert(1 << kRoundShift == kQuadTokens * kWave, "a round of a wave");

struct Range {
    int64_t lo, hi;
};
// Sequence b's positions, within the arrays whatever the offsets hold.
__device__ __forceinline__ Range range_of(const Sequences &s, int64_t b)
{
    const int64_t lo = min(max(s.offsets[b], int64_t(0)), s.n_tokens);
    return {lo, max(lo, min(s.offsets[b + 1], s.n_tokens))};
}
__device__ __forceinline__ double weight_of(const Sequences &s, int64_t targets)
{
    return s.mode == ZERO_SEQUENCE_SUM || targets == 0 ? 1.0 : 1.0 / (double)targets;
}

typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
typedef long i64x2 __attribute__((ext_vector_type(2)));
typedef i64x2 i64x2_at8 __attribute__((aligned(8)));

// N arrays' values at four neighbouring positions, and their tokens.  All loads are
// issued before any value is used: whole quads where the array has them (neighbours'
// positions too; what is outside the range is not used).
template <int N>
struct Quad {
    f32x4 x[N];
    i64x2 token[2];
    __device__ __forceinline__ Quad(const Sequences &s, const float *const (&p)[N], int64_t t, const Range &r)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = f32x4{0, 0, 0, 0};
        token[0] = token[1] = i64x2{0, 0};
        if (t >= r.hi || t + kQuadTokens <= r.lo)
            return;
        if (t + kQuadTokens <= s.n_tokens) {
            if (s.tokens) {
                token[0] = *reinterpret_cast<const i64x2_at8 *>(s.tokens + t);
                token[1] = *reinterpret_cast<const i64x2_at8 *>(s.tokens + t + 2);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (p[i])
                    x[i] = *reinterpret_cast<const f32x4_at4 *>(p[i] + t);
        } else {
#pragma unroll
            for (int k = 0; k < kQuadTokens; ++k)
                if (t + k < s.n_tokens) {
                    if (s.tokens)
                        token[k / 2][k % 2] = s.tokens[t + k];
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (p[i])
                            x[i][k] = p[i][t + k];
                }
        }
    }
    // Which of the positions are targets of the range, as bits.
    __device__ __forceinline__ unsigned targets(int64_t t, const Range &r) const
    {
        const int from = (int)min(max(r.lo - t, int64_t(0)), int64_t(kQuadTokens));
        const int to = (int)min(max(r.hi - t, int64_t(0)), int64_t(kQuadTokens));
        unsigned on = 0;
#pragma unroll
        for (int k = 0; k < kQuadTokens; ++k)
            on |= (unsigned)(k >= from && k < to && token[k / 2][k % 2] >= 0) << k;
        return on;
    }
};
__device__ __forceinline__ unsigned targets_of(const Sequences &s, int64_t t, const Range &r)
{
    const float *const none[1] = {nullptr};
    return Quad<1>(s, none, t, r).targets(t, r);
}

__device__ __forceinline__ void store_quad(float *p, int64_t t, const Range &r, const float (&x)[kQuadTokens])
{
    if (t >= r.lo && t + kQuadTokens <= r.hi) {
        *reinterpret_cast<f32x4_at4 *>(p + t) = f32x4{x[0], x[1], x[2], x[3]};
        return;
    }
#pragma unroll
    for (int k = 0; k < kQuadTokens; ++k)
        if (t + k >= r.lo && t + k < r.hi)
            p[t + k] = x[k];
}
// What a quad of the gradient holds, zeros outside the range.
__device__ __forceinline__ void load_quad(const float *p, int64_t t, const Range &r, float (&x)[kQuadTokens])
{
    if (t >= r.lo && t + kQuadTokens <= r.hi) {
        const f32x4 v = *reinterpret_cast<const f32x4_at4 *>(p + t);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        return;
    }
#pragma unroll
    for (int k = 0; k < kQuadTokens; ++k)
        x[k] = t + k >= r.lo && t + k < r.hi ? p[t + k] : 0.0f;
}

// -- sums -----------------------------------------------------------------------------

__device__ __forceinline__ void add(SequencePart &p, const SequencePart &q)
{
    p.a += q.a;
    p.b += q.b;
    p.cut += q.cut;
    p.targets += q.targets;
}
// Over a wave, in every lane, in a fixed order.
__device__ __forceinline__ SequencePart wave_total(SequencePart p)
{
#pragma unroll
    for (int off = kWave / 2; off >= 1; off >>= 1)
        add(p, SequencePart{__shfl_xor(p.a, off, kWave), __shfl_xor(p.b, off, kWave), __shfl_xor(p.cut, off, kWave),
                            __shfl_xor(p.targets, off, kWave)});
    return p;
}
// Over `waves` waves from wave `first` of a workgroup on, in their threads; `sh`: one
// per wave of the workgroup.
__device__ __forceinline__ SequencePart waves_total(SequencePart p, SequencePart *sh, int first, int waves)
{
    p = wave_total(p);
    if (threadIdx.x % kWave == 0)
        sh[threadIdx.x / kWave] = p;
    __syncthreads();
    p = sh[first];
    for (int w = 1; w < waves; ++w)
        add(p, sh[first + w]);
    return p;
}

// The share that a slot holds: sequence b's positions of a tile.
struct Share {
    int64_t b, tile;
    Range seq, part;
    bool first;   // of its sequence (of an empty sequence: the only one, empty)
    bool none;
};
__device__ __forceinline__ Share share_of(const Sequences &s, int64_t slot)
{
    const int shift = s.cut.shift, lane = threadIdx.x % kWave;
    auto start = [&](int64_t b) { return min(max(s.offsets[b], int64_t(0)), s.n_tokens); };
    // the last sequence whose first slot is not behind this one: 64 candidates at a
    // time, at the end neighbours (one less, with the start of the one behind them)
    int64_t lo = 0, n = s.n;
    while (n > kWave - 1) {
        const int64_t step = (n + kWave - 1) / kWave, c = lo + lane * step;
        const uint64_t not_behind = __ballot(c < lo + n && (start(c) >> shift) + c <= slot);
        const int k = 63 - __builtin_clzll(not_behind | 1);
        n = min(step, n - k * step);
        lo += k * step;
    }
    const int64_t own = start(min(lo + lane, s.n)), c = lo + lane;
    const uint64_t not_behind = __ballot(lane < n && (own >> shift) + c <= slot);
    const int k = 63 - __builtin_clzll(not_behind | 1);
    Share h;
    h.b = lo + k;
    h.tile = slot - h.b;
    h.seq.lo = __shfl(own, k, kWave);
    h.seq.hi = max(h.seq.lo, (int64_t)__shfl(own, k + 1, kWave));
    const int64_t begin = h.seq.lo >> shift;
    h.first = h.tile == begin;
    h.part.lo = max(h.seq.lo, h.tile << shift);
    h.part.hi = min(h.seq.hi, (h.tile + 1) << shift);
    h.none = !h.first && (h.tile < begin || h.part.lo >= h.part.hi);
    return h;
}
// A lane's part of the sums of a sequence's shares.
__device__ __forceinline__ SequencePart parts_of(const Sequences &s, int64_t b, const Range &r)
{
    SequencePart p{};
    if (r.hi > r.lo) {
        const int64_t first = (r.lo >> s.cut.shift) + b, last = ((r.hi - 1) >> s.cut.shift) + b;
        for (int64_t i = first + threadIdx.x % kWave; i <= last; i += kWave)
            add(p, s.parts[i]);
    }
    return p;
}

// -- policy ---------------------------------------------------------------------------

// e^x, e^x - 1 and e^x - 1 - x: x = n ln 2 + f, |f| <= ln(2) / 2, and the exponential's
// series in f to its 11th power.  The rest is below 2^-46 of e^x, 2^-44 of e^x - 1 and
// 2^-42 of e^x - 1 - x, which are rounded to binary32 in the end (2^-24).  A third of the
// library functions' time, which weighed more than the memory's.  Where n = 0 the last two
// are the series without its first terms, and nothing cancels.
struct Exponential {
    double e, less1, rest;
};
__device__ __forceinline__ Exponential exponential(double x)
{
    constexpr double kLog2E = 1.4426950408889634074;
    constexpr double kLn2Hi = 0x1.62e42fefa39efp-1, kLn2Lo = 0x1.abc9e3b39803fp-56;
    const double y = x > 800.0 ? 800.0 : x < -800.0 ? -800.0 : x;   // NaN stays
    const double n = __builtin_rint(y * kLog2E);
    const double f = __builtin_fma(-n, kLn2Lo, __builtin_fma(-n, kLn2Hi, y));
    double q = 1.0 / 39916800.0;
    q = __builtin_fma(q, f, 1.0 / 3628800.0);
    q = __builtin_fma(q, f, 1.0 / 362880.0);
    q = __builtin_fma(q, f, 1.0 / 40320.0);
    q = __builtin_fma(q, f, 1.0 / 5040.0);
    q = __builtin_fma(q, f, 1.0 / 720.0);
    q = __builtin_fma(q, f, 1.0 / 120.0);
    q = __builtin_fma(q, f, 1.0 / 24.0);
    q = __builtin_fma(q, f, 1.0 / 6.0);
    q = __builtin_fma(q, f, 0.5);
    const double rest = f * f * q;
    Exponential r;
    r.e = __builtin_ldexp(1.0 + (f + rest), (int)n);
    r.less1 = n == 0.0 ? f + rest : r.e - 1.0;
    r.rest = n == 0.0 ? rest : r.less1 - x;
    return r;
}

struct Term {
    double loss, kl, slope;
    int cut;
};
__device__ __forceinline__ Term policy_term(const PolicyArgs &a, float lp, float old, float ref, float adv)
{
    const double d = (double)lp - (double)old, A = adv;
    const double r = exponential(d).e;
    const bool above = A > 0.0 && d > a.log_high, below = A < 0.0 && d < a.log_low;
    Term t;
    t.cut = above || below;
    t.loss = -A * (above ? a.high : below ? a.low : r);
    t.slope = t.cut ? 0.0 : -A * r;
    t.kl = 0.0;
    if (a.ref_logprob) {
        const double x = (double)ref - (double)lp;
        const Exponential e = exponential(x);
        t.kl = x == __builtin_inf() ? x : e.rest;
        if (a.kl_coef != 0.0) {
            t.loss += a.kl_coef * t.kl;
            t.slope -= a.kl_coef * e.less1;
        }
    }
    return t;
}

// Four positions of sequence b: their sums, their slopes (0 where there is no target).
__device__ __forceinline__ void policy_quad(const PolicyArgs &a, int64_t b, int64_t t, const Range &r, SequencePart &sum,
                                            double (&slope)[kQuadTokens])
{
    const float *const arrays[4] = {a.logprob, a.old_logprob, a.ref_logprob, a.per_token ? a.advantage : nullptr};
    const Quad<4> q(a.seq, arrays, t, r);
    const float adv = a.per_token ? 0.0f : a.advantage[b];
    const unsigned on = q.targets(t, r);
#pragma unroll
    for (int k = 0; k < kQuadTokens; ++k) {
        slope[k] = 0.0;
        if (on >> k & 1) {
            const Term m = policy_term(a, q.x[0][k], q.x[1][k], q.x[2][k], a.per_token ? q.x[3][k] : adv);
            add(sum, SequencePart{m.loss, m.kl, m.cut, 1});
            slope[k] = m.slope;
        }
    }
}
// A quad's gradients: up times the slopes, zero where there is no target, whatever up is.
__device__ __forceinline__ void put_slopes(const PolicyArgs &a, int64_t t, const Range &r, double up,
                                           const double (&slope)[kQuadTokens])
{
    const bool plain = __builtin_fabs(up) < __builtin_inf();
    const unsigned on = plain ? 15u : targets_of(a.seq, t, r);
    float g[kQuadTokens];
#pragma unroll
    for (int k = 0; k < kQuadTokens; ++k)
        g[k] = on >> k & 1 ? (float)(up * slope[k]) : 0.0f;
    store_quad(a.d_logprob, t, r, g);
}
// A quad's gradients of a mean from what the first pass wrote of them, d_loss times the
// slopes: w times these (w <= 1, so digits that the first rounding below the normal range
// dropped are not missed).  One that binary32 could not hold there, though w of it may
// fit, is computed again from its target.
__device__ __forceinline__ void put_means(const PolicyArgs &a, int64_t b, int64_t t, const Range &r, double w,
                                          const float (&g)[kQuadTokens])
{
    float v[kQuadTokens];
    bool held = true;
#pragma unroll
    for (int k = 0; k < kQuadTokens; ++k) {
        v[k] = (float)(w * g[k]);
        held = held && !__builtin_isinf(g[k]);
    }
    if (!held) {
#pragma unroll
        for (int k = 0; k < kQuadTokens; ++k)
            if (__builtin_isinf(g[k])) {
                const Term m = policy_term(a, a.logprob[t + k], a.old_logprob[t + k],
                                           a.ref_logprob ? a.ref_logprob[t + k] : 0.0f,
                                           a.advantage[a.per_token ? t + k : b]);
                v[k] = (float)(w * a.d_loss[b] * m.slope);
            }
    }
    store_quad(a.d_logprob, t, r, v);
}
__device__ __forceinline__ void put_policy(const PolicyArgs &a, int64_t b, const SequencePart &p)
{
    const double w = weight_of(a.seq, p.targets);
    if (a.loss)
        a.loss[b] = (float)(w * p.a);
    if (a.kl)
        a.kl[b] = (float)(w * p.b);
    if (a.clipped)
        a.clipped[b] = p.cut;
}

// A workgroup of NT threads to a sequence; up to 4 NT positions are read once.
template <int NT>
__global__ __launch_bounds__(NT) void policy_kernel(PolicyArgs a)
{
    __shared__ SequencePart sh[NT / kWave];
    const int64_t b = blockIdx.x;
    const Range r = range_of(a.seq, b);
    const int64_t t0 = r.lo / kQuadTokens * kQuadTokens + threadIdx.x * kQuadTokens;
    const bool mean = a.seq.mode == ZERO_SEQUENCE_MEAN;
    const double d_loss = a.d_logprob ? a.d_loss[b] : 0.0;
    SequencePart sum{};
    double held[kQuadTokens], slope[kQuadTokens];
    policy_quad(a, b, t0, r, sum, held);
    for (int64_t t = t0 + NT * kQuadTokens; t < r.hi; t += NT * kQuadTokens) {
        policy_quad(a, b, t, r, sum, slope);
        if (a.d_logprob)   // a mean's are scaled below, by the same thread
            put_slopes(a, t, r, d_loss, slope);
    }
    sum = waves_total(sum, sh, 0, NT / kWave);
    if (threadIdx.x == 0)
        put_policy(a, b, sum);
    if (!a.d_logprob)
        return;
    const double w = weight_of(a.seq, sum.targets);
    put_slopes(a, t0, r, w * d_loss, held);
    for (int64_t t = t0 + NT * kQuadTokens; mean && t < r.hi; t += NT * kQuadTokens) {
        float g[kQuadTokens];
        load_quad(a.d_logprob, t, r, g);
        put_means(a, b, t, r, w, g);
    }
}

// A wave to a share: its sums; gradients of sums are finished here, those of means
// but for the targets' number: rounded to binary32 here and once more in the second pass,
// which would otherwise read the inputs and compute the terms again (300 sequences of
// 3400: 14.8 us, so 17.6; 4000 of 4000: 132, 192).
__global__ __launch_bounds__(kBlock) void policy_share_kernel(PolicyArgs a)
{
    const int64_t slot = (int64_t)blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (slot >= a.seq.cut.slots)
        return;
    const Share h = share_of(a.seq, slot);
    if (h.none || h.part.lo >= h.part.hi)
        return;
    const double d_loss = a.d_logprob ? a.d_loss[h.b] : 0.0;
    const int64_t begin = h.tile << a.seq.cut.shift;
    const int rounds = 1 << (a.seq.cut.shift - kRoundShift);
    SequencePart sum{};
    for (int i = 0; i < rounds; ++i) {
        const int64_t t = begin + (int64_t)(i * kWave + threadIdx.x % kWave) * kQuadTokens;
        double slope[kQuadTokens];
        policy_quad(a, h.b, t, h.part, sum, slope);
        if (a.d_logprob)
            put_slopes(a, t, h.part, d_loss, slope);
    }
    sum = wave_total(sum);
    if (threadIdx.x % kWave == 0)
        a.seq.parts[slot] = sum;
}
__global__ __launch_bounds__(kBlock) void policy_join_kernel(PolicyArgs a)
{
    const int64_t slot = (int64_t)blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (slot >= a.seq.cut.slots)
        return;
    const Share h = share_of(a.seq, slot);
    const bool scale = a.d_logprob && a.seq.mode == ZERO_SEQUENCE_MEAN && h.part.lo < h.part.hi;
    if (h.none || !(h.first || scale))
        return;
    // the first round's gradients are on their way while the parts are added up
    const int64_t t0 = (h.tile << a.seq.cut.shift) + threadIdx.x % kWave * kQuadTokens;
    float g[kQuadTokens];
    if (scale)
        load_quad(a.d_logprob, t0, h.part, g);
    const SequencePart sum = wave_total(parts_of(a.seq, h.b, h.seq));
    if (h.first && threadIdx.x % kWave == 0)
        put_policy(a, h.b, sum);
    if (!scale)
        return;
    const double w = weight_of(a.seq, sum.targets);
    const int rounds = 1 << (a.seq.cut.shift - kRoundShift);
    for (int i = 0; i < rounds; ++i) {
        const int64_t t = t0 + (int64_t)i * kWave * kQuadTokens;
        if (i > 0)
            load_quad(a.d_logprob, t, h.part, g);
        put_means(a, h.b, t, h.part, w, g);
    }
}

// -- preference -----------------------------------------------------------------------

// A pair's loss, and `up` times beta times its derivative by h.
__device__ __forceinline__ double preference_loss(const PreferenceArgs &a, double h)
{
    if (a.kind == ZERO_PREFER_SIGMOID) {
        // ln(1 + e^v) = max(v, 0) + ln(1 + e^-|v|); of an infinite h too
        const double near = log1p(exp(-fabs(h))), eps = a.smoothing;
        const double up = fmax(h, 0.0) + near, down = fmax(-h, 0.0) + near;
        return h != h ? h : eps == 0.0 ? down : eps == 1.0 ? up : (1.0 - eps) * down + eps * up;
    }
    if (a.kind == ZERO_PREFER_HINGE)
        return h >= 1.0 ? 0.0 : 1.0 - h;
    const double u = (h - 0.5) / a.beta;
    return u * u;
}
__device__ __forceinline__ double preference_slope(const PreferenceArgs &a, double h, double up)
{
    if (a.kind == ZERO_PREFER_SQUARED)   // beta's square may have no binary64 value
        return up * (2.0 * (h - 0.5) / a.beta);
    double slope;
    if (a.kind == ZERO_PREFER_HINGE) {
        slope = h >= 1.0 ? 0.0 : h != h ? h : -1.0;
    } else {
        // 1 / (1 + e^h) = e^-h / (1 + e^-h): of the smaller exponential, which is finite
        const double e = exponential(-fabs(h)).e, less = e / (1.0 + e), more = 1.0 / (1.0 + e);
        slope = h >= 0.0 ? a.smoothing * more - (1.0 - a.smoothing) * less
                         : a.smoothing * less - (1.0 - a.smoothing) * more;
    }
    return up * slope * a.beta;
}

__device__ __forceinline__ unsigned ratio_quad(const PreferenceArgs &a, int64_t t, const Range &r, SequencePart &sum)
{
    const float *const arrays[2] = {a.logprob, a.ref_logprob};
    const Quad<2> q(a.seq, arrays, t, r);
    const unsigned on = q.targets(t, r);
#pragma unroll
    for (int k = 0; k < kQuadTokens; ++k)
        if (on >> k & 1)
            add(sum, SequencePart{(double)q.x[0][k] - (double)q.x[1][k], 0.0, 0, 1});
    return on;
}
__device__ __forceinline__ void put_constant(const PreferenceArgs &a, int64_t t, const Range &r, unsigned on, float g)
{
    float v[kQuadTokens];
#pragma unroll
    for (int k = 0; k < kQuadTokens; ++k)
        v[k] = on >> k & 1 ? g : 0.0f;
    store_quad(a.d_logprob, t, r, v);
}
// Pair p from its sequences' sums, as log ratios and targets: lane `put` writes its loss
// and rewards, every lane gets the gradient of the chosen (of the rejected) sequence's
// targets.  `writes`: the same in every lane, whether one of them puts.
__device__ __forceinline__ float pair_gradient(const PreferenceArgs &a, int64_t p, double chosen, int chosen_targets,
                                               double rejected, int rejected_targets, bool writes, bool put,
                                               bool of_rejected)
{
    const double wc = weight_of(a.seq, chosen_targets), wr = weight_of(a.seq, rejected_targets);
    const double rc = a.beta * (chosen * wc), rr = a.beta * (rejected * wr);
    const double h = rc - rr - a.margin;
    if (writes) {
        const double loss = preference_loss(a, h);
        if (put) {
            if (a.loss)
                a.loss[p] = (float)loss;
            if (a.reward)
                a.reward[p] = (float)rc, a.reward[p + a.pairs] = (float)rr;
        }
    }
    if (!a.d_logprob)
        return 0.0f;
    const double up = preference_slope(a, h, a.d_loss[p]);
    return (float)(of_rejected ? -up * wr : up * wc);
}

// A workgroup of NT threads to a pair, half of them to each sequence; up to 2 NT
// positions of a sequence are read once.
template <int NT>
__global__ __launch_bounds__(NT) void preference_kernel(PreferenceArgs a)
{
    constexpr int Half = NT / 2, Waves = Half / kWave;
    __shared__ SequencePart sh[2 * Waves], both[2];
    const int64_t p = blockIdx.x;
    const int side = threadIdx.x / Half;
    const Range r = range_of(a.seq, p + side * a.pairs);
    const int64_t t0 = r.lo / kQuadTokens * kQuadTokens + threadIdx.x % Half * kQuadTokens;
    SequencePart sum{};
    const unsigned held = ratio_quad(a, t0, r, sum);
    for (int64_t t = t0 + Half * kQuadTokens; t < r.hi; t += Half * kQuadTokens)
        ratio_quad(a, t, r, sum);
    sum = waves_total(sum, sh, side * Waves, Waves);
    if (threadIdx.x % Half == 0)
        both[side] = sum;
    __syncthreads();
    const float g = pair_gradient(a, p, both[0].a, both[0].targets, both[1].a, both[1].targets, threadIdx.x < kWave,
                                  threadIdx.x == 0, side == 1);
    if (!a.d_logprob)
        return;
    put_constant(a, t0, r, held, g);
    for (int64_t t = t0 + Half * kQuadTokens; t < r.hi; t += Half * kQuadTokens)
        put_constant(a, t, r, targets_of(a.seq, t, r), g);
}

__global__ __launch_bounds__(kBlock) void preference_share_kernel(PreferenceArgs a)
{
    const int64_t slot = (int64_t)blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (slot >= a.seq.cut.slots)
        return;
    const Share h = share_of(a.seq, slot);
    if (h.none || h.part.lo >= h.part.hi)
        return;
    const int64_t begin = h.tile << a.seq.cut.shift;
    const int rounds = 1 << (a.seq.cut.shift - kRoundShift);
    SequencePart sum{};
    for (int i = 0; i < rounds; ++i)
        ratio_quad(a, begin + (int64_t)(i * kWave + threadIdx.x % kWave) * kQuadTokens, h.part, sum);
    sum = wave_total(sum);
    if (threadIdx.x % kWave == 0)
        a.seq.parts[slot] = sum;
}
__global__ __launch_bounds__(kBlock) void preference_join_kernel(PreferenceArgs a)
{
    const int64_t slot = (int64_t)blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (slot >= a.seq.cut.slots)
        return;
    const Share h = share_of(a.seq, slot);
    const bool rejected = h.b >= a.pairs, put = h.first && !rejected;
    const bool write = a.d_logprob && h.part.lo < h.part.hi;
    if (h.none || !(put || write))
        return;
    const int64_t p = rejected ? h.b - a.pairs : h.b, o = rejected ? p : p + a.pairs;
    // the first round's targets are on their way while the parts are added up
    const int64_t t0 = (h.tile << a.seq.cut.shift) + threadIdx.x % kWave * kQuadTokens;
    const float *const none[1] = {nullptr};
    const Quad<1> ahead(a.seq, none, t0, h.part);
    // both sequences' sums at once: log ratios in a and b, targets in cut and targets
    const SequencePart own = parts_of(a.seq, h.b, h.seq), other = parts_of(a.seq, o, range_of(a.seq, o));
    const SequencePart both = wave_total(SequencePart{own.a, other.a, own.targets, other.targets});
    const float g = rejected ? pair_gradient(a, p, both.b, both.targets, both.a, both.cut, put,
                                             put && threadIdx.x % kWave == 0, true)
                             : pair_gradient(a, p, both.a, both.cut, both.b, both.targets, put,
                                             put && threadIdx.x % kWave == 0, false);
    if (!write)
        return;
    const int rounds = 1 << (a.seq.cut.shift - kRoundShift);
    for (int i = 0; i < rounds; ++i) {
        const int64_t t = t0 + (int64_t)i * kWave * kQuadTokens;
        put_constant(a, t, h.part, i == 0 ? ahead.targets(t, h.part) : targets_of(a.seq, t, h.part), g);
    }
}

// Threads of a workgroup that takes a sequence of `mean` positions on average; some
// are several times as long.  16384 positions of the policy (of the preference) loss, us,
// most of them the call's way to the device, with
//   sequences of     64 threads      256          512
//       8            9.3 ( 8.2)    9.1 (10.0)  15.9 (18.0)
//      16            9.2 ( 8.2)    8.9 ( 8.0)  10.0 (10.3)
//     256           12.3 (10.8)    8.9 ( 8.1)   9.2 ( 8.1)
//     819           22.7 ( 7.9)    9.5 ( 8.0)   9.0 ( 8.2)
int threads_for(int64_t mean) { return mean <= 8 ? 64 : mean <= 512 ? 256 : 512; }

unsigned share_groups(const Sequences &s)
{
    return (unsigned)((s.cut.slots + kBlock / kWave - 1) / (kBlock / kWave));
}

}  // namespace

int launch_policy_loss(const PolicyArgs &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (a.seq.cut.slots > 0) {
        hipLaunchKernelGGL(policy_share_kernel, dim3(share_groups(a.seq)), dim3(kBlock), 0, st, a);
        hipLaunchKernelGGL(policy_join_kernel, dim3(share_groups(a.seq)), dim3(kBlock), 0, st, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)a.seq.n);
    switch (threads_for(a.seq.n_tokens / a.seq.n)) {
    case 64: hipLaunchKernelGGL((policy_kernel<64>), grid, dim3(64), 0, st, a); break;
    case 256: hipLaunchKernelGGL((policy_kernel<256>), grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL((policy_kernel<512>), grid, dim3(512), 0, st, a);
    }
    return hipGetLastError();
}

int launch_preference_loss(const PreferenceArgs &a, void *stream)
{
    hipStream_t st = reinterpret_cast<hipStream_t>(stream);
    if (a.seq.cut.slots > 0) {
        hipLaunchKernelGGL(preference_share_kernel, dim3(share_groups(a.seq)), dim3(kBlock), 0, st, a);
        hipLaunchKernelGGL(preference_join_kernel, dim3(share_groups(a.seq)), dim3(kBlock), 0, st, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)a.pairs);
    switch (threads_for(a.seq.n_tokens / a.seq.n)) {
    case 64: hipLaunchKernelGGL((preference_kernel<128>), grid, dim3(128), 0, st, a); break;
    case 256: hipLaunchKernelGGL((preference_kernel<512>), grid, dim3(512), 0, st, a); break;
    default: hipLaunchKernelGGL((preference_kernel<1024>), grid, dim3(1024), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace zero
