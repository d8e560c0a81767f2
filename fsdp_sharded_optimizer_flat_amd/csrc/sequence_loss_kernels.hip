// sequence_loss_kernels.hip -- losses over packed sequences of tokens' log
// probabilities: the clipped policy loss with a KL term and the preference loss
// over pairs, with their gradients.
//
// All terms are binary64: a difference of two binary32 log probabilities is exact
// there, so whether a ratio is beyond the clipping border is decided on
// logprob - old against the border's logarithm, exp(x) - 1 - x (about x^2 / 2, x often
// 10^-3) keeps its digits, and sums over long sequences lose nothing.
#include "device_common.h"
#include "sequence_loss.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kSeqBlock = 256;

struct Range {
    int64_t lo, hi;
};
// Sequence b's positions, within the arrays whatever the offsets hold.
__device__ __forceinline__ Range range_of(const Sequences &s, int64_t b)
{
    const int64_t lo = min(max(s.offsets[b], int64_t(0)), s.n_tokens);
    return {lo, max(lo, min(s.offsets[b + 1], s.n_tokens))};
}
__device__ __forceinline__ bool is_target(const Sequences &s, int64_t t)
{
    return !s.tokens || s.tokens[t] >= 0;
}
__device__ __forceinline__ double weight_of(const Sequences &s, int64_t targets)
{
    return s.mode == ZERO_SEQUENCE_SUM || targets == 0 ? 1.0 : 1.0 / (double)targets;
}

// The sum over the workgroup's threads, in every thread, in a fixed order.
template <typename T>
__device__ __forceinline__ T block_sum(T x)
{
    __shared__ T sh[kSeqBlock / kWave];
#pragma unroll
    for (int off = kWave / 2; off >= 1; off >>= 1)
        x += __shfl_xor(x, off, kWave);
    __syncthreads();
    if (threadIdx.x % kWave == 0)
        sh[threadIdx.x / kWave] = x;
    __syncthreads();
    x = sh[0];
#pragma unroll
    for (int w = 1; w < kSeqBlock / kWave; ++w)
        x += sh[w];
    return x;
}

struct Term {
    double loss, kl, slope;
    int cut;
};
__device__ __forceinline__ Term policy_term(const PolicyArgs &a, float lp, float old, float ref, float adv)
{
    const double d = (double)lp - (double)old, A = adv;
    const double r = exp(d);
    const bool above = A > 0.0 && d > a.log_high, below = A < 0.0 && d < a.log_low;
    Term t;
    t.cut = above || below;
    t.loss = -A * (above ? a.high : below ? a.low : r);
    t.slope = t.cut ? 0.0 : -A * r;
    t.kl = 0.0;
    if (a.ref_logprob) {
        const double x = (double)ref - (double)lp, e = expm1(x);
        t.kl = x == __builtin_inf() ? x : e - x;
        if (a.kl_coef != 0.0) {
            t.loss += a.kl_coef * t.kl;
            t.slope -= a.kl_coef * e;
        }
    }
    return t;
}

// One workgroup per sequence.
__global__ __launch_bounds__(kSeqBlock) void policy_kernel(PolicyArgs a)
{
    const int64_t b = blockIdx.x;
    const Range s = range_of(a.seq, b);
    const float adv = a.per_token ? 0.0f : a.advantage[b];
    int targets = 0;
    for (int64_t t = s.lo + threadIdx.x; t < s.hi; t += kSeqBlock)
        targets += is_target(a.seq, t);
    targets = block_sum(targets);
    const double w = weight_of(a.seq, targets);
    const double up = a.d_logprob ? w * (double)a.d_loss[b] : 0.0;
    double loss = 0.0, kl = 0.0;
    int cut = 0;
    for (int64_t t = s.lo + threadIdx.x; t < s.hi; t += kSeqBlock) {
        if (!is_target(a.seq, t)) {
            if (a.d_logprob)
                a.d_logprob[t] = 0.0f;
            continue;
        }
        const Term m = policy_term(a, a.logprob[t], a.old_logprob[t], a.ref_logprob ? a.ref_logprob[t] : 0.0f,
                                   a.per_token ? a.advantage[t] : adv);
        loss += m.loss;
        kl += m.kl;
        cut += m.cut;
        if (a.d_logprob)
            a.d_logprob[t] = (float)(up * m.slope);
    }
    loss = block_sum(loss);
    kl = block_sum(kl);
    cut = block_sum(cut);
    if (threadIdx.x == 0) {
        if (a.loss)
            a.loss[b] = (float)(w * loss);
        if (a.kl)
            a.kl[b] = (float)(w * kl);
        if (a.clipped)
            a.clipped[b] = cut;
    }
}

// A pair's loss and its derivative by h.
__device__ __forceinline__ void preference(const PreferenceArgs &a, double h, double &loss, double &slope)
{
    if (a.kind == ZERO_PREFER_SIGMOID) {
        // ln(1 + e^v) = max(v, 0) + ln(1 + e^-|v|); of an infinite h too
        const double near = log1p(exp(-fabs(h))), eps = a.smoothing;
        const double up = fmax(h, 0.0) + near, down = fmax(-h, 0.0) + near;
        loss = eps == 0.0 ? down : eps == 1.0 ? up : (1.0 - eps) * down + eps * up;
        slope = eps / (1.0 + exp(-h)) - (1.0 - eps) / (1.0 + exp(h));
        if (h != h)
            loss = h;
    } else if (a.kind == ZERO_PREFER_HINGE) {
        loss = h >= 1.0 ? 0.0 : 1.0 - h;
        slope = h >= 1.0 ? 0.0 : h != h ? h : -1.0;
    } else {
        const double u = (h - 0.5) / a.beta;
        loss = u * u;
        slope = 2.0 * u / a.beta;
    }
}

// One workgroup per pair.
__global__ __launch_bounds__(kSeqBlock) void preference_kernel(PreferenceArgs a)
{
    const int64_t p = blockIdx.x;
    double reward[2], w[2];
    for (int i = 0; i < 2; ++i) {
        const Range s = range_of(a.seq, p + i * a.pairs);
        double sum = 0.0;
        int targets = 0;
        for (int64_t t = s.lo + threadIdx.x; t < s.hi; t += kSeqBlock)
            if (is_target(a.seq, t)) {
                sum += a.ref_logprob ? (double)a.logprob[t] - (double)a.ref_logprob[t] : (double)a.logprob[t];
                ++targets;
            }
        w[i] = weight_of(a.seq, block_sum(targets));
        reward[i] = a.beta * (block_sum(sum) * w[i]);
        if (a.reward && threadIdx.x == 0)
            a.reward[p + i * a.pairs] = (float)reward[i];
    }
    double loss, slope;
    preference(a, reward[0] - reward[1] - a.margin, loss, slope);
    if (a.loss && threadIdx.x == 0)
        a.loss[p] = (float)loss;
    if (!a.d_logprob)
        return;
    const double up = (double)a.d_loss[p] * slope * a.beta;
    for (int i = 0; i < 2; ++i) {
        const Range s = range_of(a.seq, p + i * a.pairs);
        const float g = (float)((i ? -up : up) * w[i]);
        for (int64_t t = s.lo + threadIdx.x; t < s.hi; t += kSeqBlock)
            a.d_logprob[t] = is_target(a.seq, t) ? g : 0.0f;
    }
}

}  // namespace

int launch_policy_loss(const PolicyArgs &a, void *stream)
{
    hipLaunchKernelGGL(policy_kernel, dim3((unsigned)a.seq.n), dim3(kSeqBlock), 0,
                       reinterpret_cast<hipStream_t>(stream), a);
    return hipGetLastError();
}

int launch_preference_loss(const PreferenceArgs &a, void *stream)
{
    hipLaunchKernelGGL(preference_kernel, dim3((unsigned)a.pairs), dim3(kSeqBlock), 0,
                       reinterpret_cast<hipStream_t>(stream), a);
    return hipGetLastError();
}

}  // namespace zero
