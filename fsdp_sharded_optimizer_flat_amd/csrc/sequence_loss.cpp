// sequence_loss.cpp -- the sequence-loss entry points: argument validation,
// aliasing checks and the layout of the workspace.  Every check runs before any
// device work.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "call_check.h"
#include "sequence_loss.h"

namespace zero {
namespace {

zero_status check_sequences(const int64_t *tokens, int64_t n_tokens, const int64_t *offsets,
                            int64_t n_seqs, int32_t mode, int64_t mean, Sequences *s)
{
    if (n_tokens < 0 || n_seqs < 0 || (mode != ZERO_SEQUENCE_MEAN && mode != ZERO_SEQUENCE_SUM))
        return ZERO_EINVAL;
    if (n_tokens > ZERO_MAX_LOSS_ROWS || n_seqs > ZERO_MAX_SEQUENCES)
        return ZERO_ERANGE;
    if (n_seqs > 0 && !offsets)
        return ZERO_EINVAL;
    *s = Sequences{tokens, offsets, n_tokens, n_seqs, mode, sequence_cut(n_tokens, n_seqs, mean), nullptr};
    return ZERO_OK;
}

int64_t parts_bytes(int64_t slots) { return slots * (int64_t)sizeof(SequencePart); }

// The most slots of a call with up to n_tokens positions of up to n_seqs sequences.
int64_t most_slots(int64_t n_tokens, int64_t n_seqs)
{
    if (n_tokens <= kSequenceShort) {
        // a policy loss is cut if its sequences have more than kPolicyShort positions
        const int64_t n = std::min(n_seqs, n_tokens / (kPolicyShort + 1));
        return n > 0 ? (n_tokens >> kRoundShift) + n : 0;
    }
    // tiles of 2^shift are for as many positions as an average of 1024 tiles allows
    int64_t most = 0;
    for (int32_t shift = kRoundShift; n_seqs > 0; shift += 2) {
        const int64_t n = std::min(n_tokens, (((int64_t)1024 << shift) + 1) * n_seqs - 1);
        most = std::max(most, (n >> shift) + n_seqs);
        if (n == n_tokens)
            break;
    }
    return most;
}

// NaN is out of every range.
bool within(double x, double lo, double hi) { return x >= lo && x <= hi; }

}  // namespace

SequenceCut sequence_cut(int64_t n_tokens, int64_t n_seqs, int64_t mean)
{
    if (n_seqs == 0 || (n_tokens <= kSequenceShort && n_tokens / n_seqs <= mean))
        return {kRoundShift, 0};
    // every wave of a sequence adds up all its parts: tiles grow before an even share of
    // the positions has more than 1024 of them
    int32_t shift = kRoundShift;
    while (n_tokens / n_seqs > (int64_t)1024 << shift)
        shift += 2;
    return {shift, (n_tokens >> shift) + n_seqs};
}

}  // namespace zero

using namespace zero;

extern "C" zero_status zero_sequence_loss_workspace_bytes(int64_t n_tokens, int64_t n_seqs,
                                                          size_t *bytes)
{
    if (!bytes || n_tokens < 0 || n_seqs < 0)
        return ZERO_EINVAL;
    if (n_tokens > ZERO_MAX_LOSS_ROWS || n_seqs > ZERO_MAX_SEQUENCES)
        return ZERO_ERANGE;
    *bytes = (size_t)parts_bytes(most_slots(n_tokens, n_seqs));
    return ZERO_OK;
}

extern "C" zero_status zero_policy_loss(const float *logprob, const float *old_logprob,
                                        const float *ref_logprob, const float *advantage,
                                        int32_t per_token, const int64_t *tokens, int64_t n_tokens,
                                        const int64_t *offsets, int64_t n_seqs, double clip_low,
                                        double clip_high, double kl_coef, int32_t mode,
                                        const float *d_loss, float *loss, float *kl,
                                        int32_t *clipped, float *d_logprob, void *workspace,
                                        size_t workspace_bytes, void *stream)
{
    PolicyArgs a{};
    if (zero_status s = check_sequences(tokens, n_tokens, offsets, n_seqs, mode, kPolicyShort, &a.seq))
        return s;
    if (!within(clip_low, 0.0, 1.0) || !within(clip_high, 0.0, INFINITY) ||
        !within(kl_coef, 0.0, 1.7e308) || (!ref_logprob && n_tokens > 0 && (kl || kl_coef != 0.0)))
        return ZERO_EINVAL;
    if (n_seqs > 0 && ((!advantage && (n_tokens > 0 || !per_token)) || (d_logprob && !d_loss) ||
                       (n_tokens > 0 && (!logprob || !old_logprob || (!loss && !kl && !clipped && !d_logprob)))))
        return ZERO_EINVAL;
    const int64_t need = parts_bytes(a.seq.cut.slots);
    if (zero_status s = check_workspace_bytes(workspace, workspace_bytes, need))
        return s;
    const Span in[] = {vec(logprob, n_tokens, 4), vec(old_logprob, n_tokens, 4),
                       vec(ref_logprob, n_tokens, 4), vec(advantage, per_token ? n_tokens : n_seqs, 4),
                       vec(tokens, n_tokens, 8), vec(offsets, n_seqs + 1, 8), vec(d_loss, n_seqs, 4)};
    const Span out[] = {vec(loss, n_seqs, 4), vec(kl, n_seqs, 4), vec(clipped, n_seqs, 4),
                        vec(d_logprob, n_tokens, 4), {need ? workspace : nullptr, need, 16}};
    if (zero_status s = check_spans(in, 7, out, 5))
        return s;
    if (n_seqs == 0)
        return ZERO_OK;
    a.seq.parts = static_cast<SequencePart *>(workspace);
    a.logprob = logprob;
    a.old_logprob = old_logprob;
    a.ref_logprob = ref_logprob;
    a.advantage = advantage;
    a.d_loss = d_loss;
    a.per_token = per_token;
    a.low = 1.0 - clip_low;
    a.high = 1.0 + clip_high;
    a.log_low = std::log1p(-clip_low);
    a.log_high = std::log1p(clip_high);
    a.kl_coef = kl_coef;
    a.loss = loss;
    a.kl = kl;
    a.clipped = clipped;
    a.d_logprob = d_logprob;
    return done(launch_policy_loss(a, stream), "zero_policy_loss");
}

extern "C" zero_status zero_preference_loss(const float *logprob, const float *ref_logprob,
                                            const int64_t *tokens, int64_t n_tokens,
                                            const int64_t *offsets, int64_t n_pairs, int32_t kind,
                                            double beta, double margin, double smoothing,
                                            int32_t mode, const float *d_loss, float *loss,
                                            float *reward, float *d_logprob, void *workspace,
                                            size_t workspace_bytes, void *stream)
{
    PreferenceArgs a{};
    if (n_pairs < 0)
        return ZERO_EINVAL;
    if (n_pairs > ZERO_MAX_SEQUENCES / 2)
        return ZERO_ERANGE;
    if (zero_status s = check_sequences(tokens, n_tokens, offsets, 2 * n_pairs, mode, kSequenceShort, &a.seq))
        return s;
    if ((kind != ZERO_PREFER_SIGMOID && kind != ZERO_PREFER_HINGE && kind != ZERO_PREFER_SQUARED) ||
        !std::isfinite(beta) || !(beta > 0.0) || !std::isfinite(margin) || !within(smoothing, 0.0, 1.0) ||
        (smoothing != 0.0 && kind != ZERO_PREFER_SIGMOID))
        return ZERO_EINVAL;
    if (n_pairs > 0 && ((d_logprob && !d_loss) || (n_tokens > 0 && (!logprob || (!loss && !reward && !d_logprob)))))
        return ZERO_EINVAL;
    const int64_t need = parts_bytes(a.seq.cut.slots);
    if (zero_status s = check_workspace_bytes(workspace, workspace_bytes, need))
        return s;
    const Span in[] = {vec(logprob, n_tokens, 4), vec(ref_logprob, n_tokens, 4), vec(tokens, n_tokens, 8),
                       vec(offsets, 2 * n_pairs + 1, 8), vec(d_loss, n_pairs, 4)};
    const Span out[] = {vec(loss, n_pairs, 4), vec(reward, 2 * n_pairs, 4), vec(d_logprob, n_tokens, 4),
                        {need ? workspace : nullptr, need, 16}};
    if (zero_status s = check_spans(in, 5, out, 4))
        return s;
    if (n_pairs == 0)
        return ZERO_OK;
    a.seq.parts = static_cast<SequencePart *>(workspace);
    a.logprob = logprob;
    a.ref_logprob = ref_logprob;
    a.d_loss = d_loss;
    a.pairs = n_pairs;
    a.kind = kind;
    a.beta = beta;
    a.margin = margin;
    a.smoothing = smoothing;
    a.loss = loss;
    a.reward = reward;
    a.d_logprob = d_logprob;
    return done(launch_preference_loss(a, stream), "zero_preference_loss");
}
