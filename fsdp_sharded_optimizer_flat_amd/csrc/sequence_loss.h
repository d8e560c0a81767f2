// sequence_loss.h -- what the sequence-loss entry points (sequence_loss.cpp) hand
// to the kernels (sequence_loss_kernels.hip).  Not part of the public ABI.
#pragma once

#include "zero_internal.h"

namespace zero {

// Up to kSequenceShort positions a call is one launch, a workgroup to a sequence or
// pair; the policy loss only if its sequences have at most kPolicyShort on average, which
// a workgroup of 512 reads once.  Measured, one launch against two: 16 sequences of 1024
// 9.0 : 11.4 us, one of 16384 19.1 : 12.2 (its preference loss 8.4 : 10.9), where one of
// 16 has 16000 of 16384 22 : 11.  64 of 1024 are 8.2 : 10.7, but 64 of which one has
// 60000 positions 75 : 11, and lengths are not known here: so no further.
constexpr int64_t kSequenceShort = 16384, kPolicyShort = 2048;

// Longer ones are cut into tiles of 2^shift positions, whole rounds of a wave (four
// positions to a lane); a wave takes a sequence's share of a tile.
constexpr int kRoundShift = 8;
struct SequenceCut {
    int32_t shift;
    int64_t slots;   // shares at most; 0: not cut
};
SequenceCut sequence_cut(int64_t n_tokens, int64_t n_seqs, int64_t mean);   // whole up to `mean` each

// A share's sums.  Policy: of the losses and k, targets beyond the border; preference:
// of the log ratios.
struct SequencePart {
    double a, b;
    int32_t cut, targets;
};

// The packed sequences of a call.
struct Sequences {
    const int64_t *tokens;    // NULL: every position is a target
    const int64_t *offsets;   // n + 1
    int64_t n_tokens, n;
    int32_t mode;
    SequenceCut cut;
    SequencePart *parts;      // cut.slots of them
};

struct PolicyArgs {
    Sequences seq;
    const float *logprob, *old_logprob, *ref_logprob, *advantage, *d_loss;
    int32_t per_token;
    double low, high;             // 1 - clip_low, 1 + clip_high
    double log_low, log_high;     // their logarithms
    double kl_coef;
    float *loss, *kl, *d_logprob;
    int32_t *clipped;
};
int launch_policy_loss(const PolicyArgs &a, void *stream);

struct PreferenceArgs {
    Sequences seq;                // n = 2 pairs
    const float *logprob, *ref_logprob, *d_loss;
    int64_t pairs;
    int32_t kind;
    double beta, margin, smoothing;
    float *loss, *reward, *d_logprob;
};
int launch_preference_loss(const PreferenceArgs &a, void *stream);

}  // namespace zero
