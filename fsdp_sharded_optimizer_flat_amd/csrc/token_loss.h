// token_loss.h -- what the token-loss entry points (token_loss.cpp) hand to
// the kernels (logprob_kernels.hip, distill_kernels.hip).  Not part of the public ABI.
#pragma once

#include "zero_internal.h"

namespace zero {

// Threads of a token-loss workgroup, unless it holds a row or sums one of few.
constexpr int kLossBlock = 256;

// Most elements one workgroup reduces: its bitmap of listed tokens is 16 KiB.
constexpr int64_t kLossMaxSegment = int64_t(1) << 17;

// Up to this many rows of at most kLossWideVocab elements are not cut: a workgroup
// of 1024 threads sums each.
constexpr int64_t kLossWideRows = 256, kLossWideVocab = int64_t(1) << 16;

// The rows of a call: `logits` in rows of `stride` elements, `vocab` used.
struct LossRows {
    const void *logits;
    int64_t stride;
    int64_t rows;
    int32_t vocab;
    int32_t dtype;
    float scale;
    float c;    // scale * log2(e), rounded once: logits are compared in binary logarithms
};

// The workgroups a row of a forward pass is cut for.
int32_t loss_segments(int64_t rows, int64_t vocab, int32_t top_k);

// One workgroup's share of a row: the largest logit, the sum of 2^(t) and of
// t 2^t over its elements, t = c * (logit - max) (entropy).
struct LossPart {
    float m, s, a, pad;
};

struct LogprobArgs {
    LossRows in;
    const int64_t *tokens;
    float *logprob, *entropy, *stats;
    int32_t top_k;
    int32_t *top_index;
    float *top_logprob;
    bool with_entropy;   // the entropy is wanted (also where only the gradient uses it)
    LossPart *parts;     // rows * segs, where segs > 1
    uint64_t *keys;      // rows * segs * top_k, where segs > 1
};
int launch_logprob(const LogprobArgs &a, int32_t segs, void *stream);

struct LogprobGradArgs {
    LossRows in;
    const int64_t *tokens;
    const float *stats, *entropy, *d_logprob, *d_entropy;
    void *d_logits;
    int64_t d_stride;
};
int launch_logprob_grad(const LogprobGradArgs &a, void *stream);

struct DistillArgs {
    LossRows in;
    int32_t top_k, mode;
    const int32_t *top_index;
    const float *top_value;
    float *loss, *stats;
    LossPart *parts;
};
int launch_distill(const DistillArgs &a, int32_t segs, void *stream);

struct DistillGradArgs {
    LossRows in;
    int32_t top_k, mode;
    const int32_t *top_index;
    const float *top_value;
    const float *stats, *d_loss;
    void *d_logits;
    int64_t d_stride;
};
int launch_distill_grad(const DistillGradArgs &a, void *stream);

// Forward and backward in one launch, where a workgroup can hold a row.
bool logprob_row_held(const LossRows &in);
bool distill_row_held(const LossRows &in);
int launch_logprob_fused(const LogprobArgs &a, const LogprobGradArgs &b, void *stream);
int launch_distill_fused(const DistillArgs &a, const DistillGradArgs &b, void *stream);

}  // namespace zero
