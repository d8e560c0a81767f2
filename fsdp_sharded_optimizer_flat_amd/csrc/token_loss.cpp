// token_loss.cpp -- the token-loss entry points: argument validation, aliasing
// checks, the split of a row over workgroups and the layout of the workspace.
// Every check runs before any device work.
#include <hip/hip_runtime.h>

#include <cmath>

#include "token_loss.h"

namespace zero {

namespace {

constexpr double kLog2E = 1.4426950408889634074;

int esize(int32_t d) { return d == ZERO_BF16 ? 2 : 4; }

// A buffer of the call: `bytes` from p, elements of `align` bytes.
struct Span {
    const void *p;
    int64_t bytes;
    int align;
};

bool overlaps(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0)
        return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// The outputs must be aligned and apart from each other and from the inputs.
zero_status check_spans(const Span *in, int n_in, const Span *out, int n_out)
{
    for (int i = 0; i < n_in; ++i)
        if ((uintptr_t)in[i].p % (uintptr_t)in[i].align)
            return ZERO_EALIGN;
    for (int i = 0; i < n_out; ++i)
        if ((uintptr_t)out[i].p % (uintptr_t)out[i].align)
            return ZERO_EALIGN;
    for (int i = 0; i < n_out; ++i) {
        for (int k = 0; k < n_in; ++k)
            if (overlaps(out[i], in[k]))
                return ZERO_EINVAL;
        for (int k = 0; k < i; ++k)
            if (overlaps(out[i], out[k]))
                return ZERO_EINVAL;
    }
    return ZERO_OK;
}

// Sizes and the logits of a call; fills `r`.
zero_status check_rows(const void *logits, int32_t dtype, int64_t rows, int64_t vocab,
                       int64_t row_stride, float scale, LossRows *r)
{
    if ((dtype != ZERO_F32 && dtype != ZERO_BF16) || rows < 0 || vocab < 1 ||
        row_stride < vocab || !std::isfinite(scale) || !(scale > 0.0f))
        return ZERO_EINVAL;
    if (vocab > ZERO_MAX_VOCAB || rows > ZERO_MAX_LOSS_ROWS ||
        row_stride > (int64_t(1) << 61) / 4 / (rows > 0 ? rows : 1) || scale < 0x1p-20f ||
        scale > 0x1p20f)
        return ZERO_ERANGE;
    if (!logits && rows > 0)
        return ZERO_EINVAL;
    r->logits = logits;
    r->stride = row_stride;
    r->rows = rows;
    r->vocab = (int32_t)vocab;
    r->dtype = dtype;
    r->scale = scale;
    r->c = (float)((double)scale * kLog2E);
    return ZERO_OK;
}

Span matrix(const void *p, const LossRows &r, int64_t stride)
{
    const int es = esize(r.dtype);
    return {p, r.rows > 0 ? ((r.rows - 1) * stride + r.vocab) * es : 0, es};
}
Span logits_span(const LossRows &r) { return matrix(r.logits, r, r.stride); }
Span vec(const void *p, int64_t n, int es) { return {p, p ? n * es : 0, es}; }

// The gradient may be written over the logits, row for row, but must not
// overlap them otherwise.
bool in_place(const LossRows &r, const void *d_logits, int64_t d_stride)
{
    return d_logits == r.logits && d_stride == r.stride;
}

// A call's workspace: the fused calls' row statistics, then the partial
// results of split rows, then their top keys.
struct Workspace {
    int64_t stats = 0, entropy = 0, parts = 0, keys = 0, bytes = 0;
};
int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }
Workspace workspace_layout(int64_t rows, int32_t segs, int32_t top_k, bool fused)
{
    Workspace w;
    int64_t at = 0;
    if (fused) {
        w.stats = at;
        at = up16(at + rows * 4 * (int64_t)sizeof(float));
        w.entropy = at;
        at = up16(at + rows * (int64_t)sizeof(float));
    }
    if (segs > 1) {
        w.parts = at;
        at = up16(at + rows * segs * (int64_t)sizeof(LossPart));
        w.keys = at;
        at = up16(at + rows * segs * top_k * (int64_t)sizeof(uint64_t));
    }
    w.bytes = at;
    return w;
}

zero_status check_workspace(const void *ws, size_t have, const Workspace &w)
{
    if (w.bytes == 0)
        return ZERO_OK;
    if (!ws)
        return ZERO_EINVAL;
    if ((uintptr_t)ws % 16)
        return ZERO_EALIGN;
    return have < (size_t)w.bytes ? ZERO_ENOSPC : ZERO_OK;
}

char *at(void *ws, int64_t off) { return static_cast<char *>(ws) + off; }

zero_status done(int e, const char *where) { return e == hipSuccess ? ZERO_OK : hip_fail(e, where); }

}  // namespace

int32_t loss_segments(int64_t rows, int64_t vocab, int32_t top_k)
{
    // One workgroup per row keeps the whole chip busy from about 1024 rows on
    // (4 workgroups on each of 256 compute units).  Fewer rows are cut so that
    // there are about that many workgroups, in segments of at least 2048 elements
    // and 128 per wanted alternative, with at most 4096 alternatives for the joining
    // workgroup.  Up to 256 rows of at most 65536 elements stay whole: a workgroup of
    // 1024 threads sums a row sooner than a second launch joins its segments, except
    // for few long rows without many alternatives (bf16, whole and cut, us):
    //     rows x elements   entropy    and top 5    and top 20   distillation, 64 listed
    //       1 x  20000     5.6   6.4    8.7  10.1    9.1  10.5     6.3  13.2
    //       1 x  50304     7.6   6.6   11.6  11.3   11.9  12.4     8.2  13.3
    //       1 x  65536     8.0   6.4   12.5  12.0   12.8  12.7     9.3  13.2
    //      16 x  50304     8.3   7.5   12.5  12.6   12.7  13.8     8.9  14.2
    //      64 x  20000     6.9   7.9   10.0  12.1   10.3  12.3     7.4  15.2
    //      64 x  65536     9.0   9.0   13.9  14.0   15.1  16.2    10.7  16.0
    //     256 x  50304    10.2  12.5   14.5  17.6   15.2  19.7    11.2  19.5
    // There is one border for all calls; where cut rows win it costs up to 1.6 us.  A
    // function of the sizes alone, so the result does not depend on the device's
    // state.
    if (rows <= kLossWideRows && vocab <= kLossWideVocab)
        return 1;
    const int64_t need = (vocab + kLossMaxSegment - 1) / kLossMaxSegment;
    int64_t segs = rows > 0 ? (1024 + rows - 1) / rows : 1;
    const int64_t least = top_k > 16 ? 128 * (int64_t)top_k : 2048;
    if (segs > vocab / least)
        segs = vocab / least;
    if (top_k > 0 && segs > 4096 / top_k)
        segs = 4096 / top_k;
    if (segs < need)
        segs = need;
    if (segs < 1)
        segs = 1;
    return (int32_t)segs;
}

}  // namespace zero

using namespace zero;

extern "C" zero_status zero_loss_workspace_bytes(int64_t rows, int64_t vocab, int32_t top_k,
                                                 size_t *bytes)
{
    if (!bytes || rows < 0 || vocab < 1 || top_k < 0)
        return ZERO_EINVAL;
    if (vocab > ZERO_MAX_VOCAB || rows > ZERO_MAX_LOSS_ROWS || top_k > ZERO_MAX_TOP)
        return ZERO_ERANGE;
    // the forward calls' split depends on top_k, the fused ones' does not; with fewer
    // alternatives a row may be cut further and need more for its partial results
    int64_t most = workspace_layout(rows, loss_segments(rows, vocab, 0), 0, true).bytes;
    for (int32_t k = 0; k <= top_k; ++k) {
        const int64_t f = workspace_layout(rows, loss_segments(rows, vocab, k), k, false).bytes;
        most = f > most ? f : most;
    }
    *bytes = (size_t)most;
    return ZERO_OK;
}

extern "C" zero_status zero_logprob(const void *logits, int32_t dtype, int64_t rows, int64_t vocab,
                                    int64_t row_stride, float scale, const int64_t *tokens,
                                    float *logprob, float *entropy, float *stats, int32_t top_k,
                                    int32_t *top_index, float *top_logprob, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    LogprobArgs a{};
    if (zero_status s = check_rows(logits, dtype, rows, vocab, row_stride, scale, &a.in))
        return s;
    if (top_k < 0 || (rows > 0 && ((logprob && !tokens) || (top_k > 0) != (top_index != nullptr) ||
                                   (top_k > 0) != (top_logprob != nullptr))))
        return ZERO_EINVAL;
    if (top_k > ZERO_MAX_TOP)
        return ZERO_ERANGE;
    if (rows > 0 && !logprob && !entropy && !stats && top_k == 0)
        return ZERO_EINVAL;
    const int32_t segs = loss_segments(rows, vocab, top_k);
    const Workspace w = workspace_layout(rows, segs, top_k, false);
    if (zero_status s = check_workspace(workspace, workspace_bytes, w))
        return s;
    const Span in[] = {logits_span(a.in), vec(tokens, rows, 8)};
    const Span out[] = {vec(logprob, rows, 4), vec(entropy, rows, 4), vec(stats, 2 * rows, 4),
                        vec(top_index, rows * top_k, 4), vec(top_logprob, rows * top_k, 4),
                        {w.bytes ? workspace : nullptr, w.bytes, 16}};
    if (zero_status s = check_spans(in, 2, out, 6))
        return s;
    if (rows == 0)
        return ZERO_OK;
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.stats = stats;
    a.top_k = top_k;
    a.top_index = top_index;
    a.top_logprob = top_logprob;
    a.with_entropy = entropy != nullptr;
    a.parts = (LossPart *)at(workspace, w.parts);
    a.keys = (uint64_t *)at(workspace, w.keys);
    return done(launch_logprob(a, segs, stream), "zero_logprob");
}

extern "C" zero_status zero_logprob_grad(const void *logits, int32_t dtype, int64_t rows,
                                         int64_t vocab, int64_t row_stride, float scale,
                                         const int64_t *tokens, const float *stats,
                                         const float *entropy, const float *d_logprob,
                                         const float *d_entropy, void *d_logits,
                                         int64_t d_row_stride, void *stream)
{
    LogprobGradArgs a{};
    if (zero_status s = check_rows(logits, dtype, rows, vocab, row_stride, scale, &a.in))
        return s;
    if (d_row_stride < vocab ||
        (rows > 0 && ((!d_logprob && !d_entropy) || (d_logprob && !tokens) ||
                      (d_entropy && !entropy) || !stats || !d_logits)))
        return ZERO_EINVAL;
    if (d_row_stride > (int64_t(1) << 61) / 4 / (rows > 0 ? rows : 1))
        return ZERO_ERANGE;
    const bool same = in_place(a.in, d_logits, d_row_stride);
    const Span in[] = {same ? Span{nullptr, 0, 1} : logits_span(a.in), vec(tokens, rows, 8),
                       vec(stats, 2 * rows, 4), vec(entropy, rows, 4), vec(d_logprob, rows, 4),
                       vec(d_entropy, rows, 4)};
    const Span out[] = {matrix(d_logits, a.in, d_row_stride)};
    if (zero_status s = check_spans(in, 6, out, 1))
        return s;
    if (rows == 0)
        return ZERO_OK;
    a.tokens = tokens;
    a.stats = stats;
    a.entropy = entropy;
    a.d_logprob = d_logprob;
    a.d_entropy = d_entropy;
    a.d_logits = d_logits;
    a.d_stride = d_row_stride;
    return done(launch_logprob_grad(a, stream), "zero_logprob_grad");
}

extern "C" zero_status zero_logprob_fused(const void *logits, int32_t dtype, int64_t rows,
                                          int64_t vocab, int64_t row_stride, float scale,
                                          const int64_t *tokens, const float *d_logprob,
                                          const float *d_entropy, float *logprob, float *entropy,
                                          void *d_logits, int64_t d_row_stride, void *workspace,
                                          size_t workspace_bytes, void *stream)
{
    LogprobArgs a{};
    if (zero_status s = check_rows(logits, dtype, rows, vocab, row_stride, scale, &a.in))
        return s;
    if (d_row_stride < vocab ||
        (rows > 0 && ((!d_logprob && !d_entropy) || ((d_logprob || logprob) && !tokens) || !d_logits)))
        return ZERO_EINVAL;
    if (d_row_stride > (int64_t(1) << 61) / 4 / (rows > 0 ? rows : 1))
        return ZERO_ERANGE;
    const bool held = logprob_row_held(a.in);
    const int32_t segs = loss_segments(rows, vocab, 0);
    const Workspace w = held ? Workspace{} : workspace_layout(rows, segs, 0, true);
    if (zero_status s = check_workspace(workspace, workspace_bytes, w))
        return s;
    const bool same = in_place(a.in, d_logits, d_row_stride);
    const Span in[] = {same ? Span{nullptr, 0, 1} : logits_span(a.in), vec(tokens, rows, 8),
                       vec(d_logprob, rows, 4), vec(d_entropy, rows, 4)};
    const Span out[] = {vec(logprob, rows, 4), vec(entropy, rows, 4),
                        matrix(d_logits, a.in, d_row_stride),
                        {w.bytes ? workspace : nullptr, w.bytes, 16}};
    if (zero_status s = check_spans(in, 4, out, 4))
        return s;
    if (rows == 0)
        return ZERO_OK;
    LogprobGradArgs g{};
    g.in = a.in;
    g.tokens = a.tokens = tokens;
    g.d_logprob = d_logprob;
    g.d_entropy = d_entropy;
    g.d_logits = d_logits;
    g.d_stride = d_row_stride;
    a.logprob = logprob;
    a.entropy = entropy;
    a.with_entropy = entropy || d_entropy;
    if (held)
        return done(launch_logprob_fused(a, g, stream), "zero_logprob_fused");
    if (d_entropy && !entropy)
        a.entropy = (float *)at(workspace, w.entropy);
    a.stats = (float *)at(workspace, w.stats);
    a.parts = (LossPart *)at(workspace, w.parts);
    if (int e = launch_logprob(a, segs, stream))
        return done(e, "zero_logprob_fused");
    g.stats = a.stats;
    g.entropy = a.entropy;
    return done(launch_logprob_grad(g, stream), "zero_logprob_fused");
}

namespace {
zero_status check_teacher(int64_t rows, int32_t top_k, const int32_t *top_index,
                          const float *top_value, int32_t mode)
{
    if (top_k < 1 || (mode != ZERO_DISTILL_RENORM && mode != ZERO_DISTILL_TAIL) ||
        (rows > 0 && (!top_index || !top_value)))
        return ZERO_EINVAL;
    return top_k > ZERO_MAX_TOP ? ZERO_ERANGE : ZERO_OK;
}
}  // namespace

extern "C" zero_status zero_distill(const void *logits, int32_t dtype, int64_t rows, int64_t vocab,
                                    int64_t row_stride, float scale, int32_t top_k,
                                    const int32_t *top_index, const float *top_value, int32_t mode,
                                    float *loss, float *stats, void *workspace,
                                    size_t workspace_bytes, void *stream)
{
    DistillArgs a{};
    if (zero_status s = check_rows(logits, dtype, rows, vocab, row_stride, scale, &a.in))
        return s;
    if (zero_status s = check_teacher(rows, top_k, top_index, top_value, mode))
        return s;
    if (rows > 0 && !loss && !stats)
        return ZERO_EINVAL;
    const int32_t segs = loss_segments(rows, vocab, 0);
    const Workspace w = workspace_layout(rows, segs, 0, false);
    if (zero_status s = check_workspace(workspace, workspace_bytes, w))
        return s;
    const Span in[] = {logits_span(a.in), vec(top_index, rows * top_k, 4),
                       vec(top_value, rows * top_k, 4)};
    const Span out[] = {vec(loss, rows, 4), vec(stats, 4 * rows, 4),
                        {w.bytes ? workspace : nullptr, w.bytes, 16}};
    if (zero_status s = check_spans(in, 3, out, 3))
        return s;
    if (rows == 0)
        return ZERO_OK;
    a.top_k = top_k;
    a.mode = mode;
    a.top_index = top_index;
    a.top_value = top_value;
    a.loss = loss;
    a.stats = stats;
    a.parts = (LossPart *)at(workspace, w.parts);
    return done(launch_distill(a, segs, stream), "zero_distill");
}

extern "C" zero_status zero_distill_grad(const void *logits, int32_t dtype, int64_t rows,
                                         int64_t vocab, int64_t row_stride, float scale,
                                         int32_t top_k, const int32_t *top_index,
                                         const float *top_value, int32_t mode, const float *stats,
                                         const float *d_loss, void *d_logits, int64_t d_row_stride,
                                         void *stream)
{
    DistillGradArgs a{};
    if (zero_status s = check_rows(logits, dtype, rows, vocab, row_stride, scale, &a.in))
        return s;
    if (zero_status s = check_teacher(rows, top_k, top_index, top_value, mode))
        return s;
    if (d_row_stride < vocab || (rows > 0 && (!stats || !d_loss || !d_logits)))
        return ZERO_EINVAL;
    if (d_row_stride > (int64_t(1) << 61) / 4 / (rows > 0 ? rows : 1))
        return ZERO_ERANGE;
    const bool same = in_place(a.in, d_logits, d_row_stride);
    const Span in[] = {same ? Span{nullptr, 0, 1} : logits_span(a.in),
                       vec(top_index, rows * top_k, 4), vec(top_value, rows * top_k, 4),
                       vec(stats, 4 * rows, 4), vec(d_loss, rows, 4)};
    const Span out[] = {matrix(d_logits, a.in, d_row_stride)};
    if (zero_status s = check_spans(in, 5, out, 1))
        return s;
    if (rows == 0)
        return ZERO_OK;
    a.top_k = top_k;
    a.mode = mode;
    a.top_index = top_index;
    a.top_value = top_value;
    a.stats = stats;
    a.d_loss = d_loss;
    a.d_logits = d_logits;
    a.d_stride = d_row_stride;
    return done(launch_distill_grad(a, stream), "zero_distill_grad");
}

extern "C" zero_status zero_distill_fused(const void *logits, int32_t dtype, int64_t rows,
                                          int64_t vocab, int64_t row_stride, float scale,
                                          int32_t top_k, const int32_t *top_index,
                                          const float *top_value, int32_t mode,
                                          const float *d_loss, float *loss, void *d_logits,
                                          int64_t d_row_stride, void *workspace,
                                          size_t workspace_bytes, void *stream)
{
    DistillArgs a{};
    if (zero_status s = check_rows(logits, dtype, rows, vocab, row_stride, scale, &a.in))
        return s;
    if (zero_status s = check_teacher(rows, top_k, top_index, top_value, mode))
        return s;
    if (d_row_stride < vocab || (rows > 0 && (!d_loss || !d_logits)))
        return ZERO_EINVAL;
    if (d_row_stride > (int64_t(1) << 61) / 4 / (rows > 0 ? rows : 1))
        return ZERO_ERANGE;
    const bool held = distill_row_held(a.in);
    const int32_t segs = loss_segments(rows, vocab, 0);
    const Workspace w = held ? Workspace{} : workspace_layout(rows, segs, 0, true);
    if (zero_status s = check_workspace(workspace, workspace_bytes, w))
        return s;
    const bool same = in_place(a.in, d_logits, d_row_stride);
    const Span in[] = {same ? Span{nullptr, 0, 1} : logits_span(a.in),
                       vec(top_index, rows * top_k, 4), vec(top_value, rows * top_k, 4),
                       vec(d_loss, rows, 4)};
    const Span out[] = {vec(loss, rows, 4), matrix(d_logits, a.in, d_row_stride),
                        {w.bytes ? workspace : nullptr, w.bytes, 16}};
    if (zero_status s = check_spans(in, 4, out, 3))
        return s;
    if (rows == 0)
        return ZERO_OK;
    a.top_k = top_k;
    a.mode = mode;
    a.top_index = top_index;
    a.top_value = top_value;
    a.loss = loss;
    DistillGradArgs g{};
    g.in = a.in;
    g.top_k = top_k;
    g.mode = mode;
    g.top_index = top_index;
    g.top_value = top_value;
    g.d_loss = d_loss;
    g.d_logits = d_logits;
    g.d_stride = d_row_stride;
    if (held)
        return done(launch_distill_fused(a, g, stream), "zero_distill_fused");
    a.stats = (float *)at(workspace, w.stats);
    a.parts = (LossPart *)at(workspace, w.parts);
    if (int e = launch_distill(a, segs, stream))
        return done(e, "zero_distill_fused");
    g.stats = a.stats;
    return done(launch_distill_grad(g, stream), "zero_distill_fused");
}
