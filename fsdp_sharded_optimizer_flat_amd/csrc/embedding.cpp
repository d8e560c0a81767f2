// embedding.cpp -- the embedding entry points: argument validation, aliasing
// checks and the layout of the gradient's workspace.  Every check runs before any
// device work.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "call_check.h"
#include "embedding.h"

namespace zero {
namespace {

struct Workspace {
    int64_t chunk_key = 0, chunk_row = 0, samples = -1, key = 0, row = 0, parts = 0, bytes = 0;
    int32_t chunk = 0, segment = 0, segments = 0, columns = 0;
};
Workspace workspace_layout(int64_t rows, int64_t hidden)
{
    Workspace w;
    w.chunk = embedding_chunk(rows);
    w.segment = embedding_segment(rows, hidden);
    w.segments = (int32_t)((rows + w.segment - 1) / w.segment);
    w.columns = (int32_t)((hidden + 7) / 8 * 8);
    const int64_t list = up16(rows * 4);
    int64_t at = 0;
    w.chunk_key = at, at += list;
    w.chunk_row = at, at += list;
    w.key = w.chunk_key, w.row = w.chunk_row;
    if (rows > w.chunk) {
        // (of small chunks: more rows never need less)
        w.samples = at, at += (rows + kSortChunk - 1) / kSortChunk * kSamples * 4;
        w.key = at, at += list;
        w.row = at, at += list;
    }
    if (w.segments > 1) {
        w.parts = at;
        at += (int64_t)w.segments * 2 * w.columns * 4;
    }
    w.bytes = at;
    return w;
}

zero_status check_sizes(int64_t rows, int64_t vocab, int64_t hidden, int64_t most_rows)
{
    if (rows < 0 || vocab < 1 || hidden < 1)
        return ZERO_EINVAL;
    return rows > most_rows || vocab > ZERO_MAX_VOCAB || hidden > ZERO_MAX_HIDDEN ? ZERO_ERANGE : ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_embedding(const void *table, int32_t dtype, int64_t vocab,
                                      int64_t hidden, int64_t row_stride, const int64_t *tokens,
                                      int64_t rows, float scale, void *out, int32_t out_dtype,
                                      int64_t out_stride, void *stream)
{
    if (bad_dtype(dtype) || bad_dtype(out_dtype) || !std::isfinite(scale))
        return ZERO_EINVAL;
    if (zero_status s = check_sizes(rows, vocab, hidden, ZERO_MAX_LOSS_ROWS))
        return s;
    if (row_stride < hidden || out_stride < hidden || (rows > 0 && (!table || !tokens || !out)))
        return ZERO_EINVAL;
    if (!stride_fits(vocab, row_stride) || !stride_fits(rows, out_stride))
        return ZERO_ERANGE;
    const Span in[] = {matrix(table, vocab, hidden, row_stride, esize(dtype)), vec(tokens, rows, 8)};
    const Span to[] = {matrix(out, rows, hidden, out_stride, esize(out_dtype))};
    if (zero_status s = check_spans(in, 2, to, 1))
        return s;
    if (rows == 0)
        return ZERO_OK;
    EmbeddingArgs a{};
    a.table = table;
    a.vocab = vocab;
    a.stride = row_stride;
    a.tokens = tokens;
    a.rows = rows;
    a.out = out;
    a.out_stride = out_stride;
    a.hidden = (int32_t)hidden;
    a.dtype = dtype;
    a.out_dtype = out_dtype;
    a.scale = scale;
    return done(launch_embedding(a, stream), "zero_embedding");
}

extern "C" zero_status zero_embedding_grad_workspace_bytes(int64_t rows, int64_t vocab,
                                                           int64_t hidden, size_t *bytes)
{
    if (!bytes)
        return ZERO_EINVAL;
    if (zero_status s = check_sizes(rows, vocab, hidden, ZERO_MAX_EMBEDDING_ROWS))
        return s;
    // longer segments have fewer parts: what serves these rows serves fewer of them too
    int64_t need = workspace_layout(rows, hidden).bytes;
    for (const int64_t work : kSegmentWork)
        need = std::max(need, workspace_layout(std::min(rows, work / embedding_slabs(hidden)), hidden).bytes);
    *bytes = (size_t)need;
    return ZERO_OK;
}

extern "C" zero_status zero_embedding_grad(const void *d_out, int32_t dtype, int64_t rows,
                                           int64_t hidden, int64_t row_stride,
                                           const int64_t *tokens, float scale, void *d_table,
                                           int32_t table_dtype, int64_t vocab,
                                           int64_t table_stride, int32_t accumulate,
                                           void *workspace, size_t workspace_bytes, void *stream)
{
    if (bad_dtype(dtype) || bad_dtype(table_dtype) || !std::isfinite(scale) ||
        (accumulate != 0 && accumulate != 1))
        return ZERO_EINVAL;
    if (zero_status s = check_sizes(rows, vocab, hidden, ZERO_MAX_EMBEDDING_ROWS))
        return s;
    if (row_stride < hidden || table_stride < hidden || !d_table || (rows > 0 && (!d_out || !tokens)))
        return ZERO_EINVAL;
    if (!stride_fits(rows, row_stride) || !stride_fits(vocab, table_stride))
        return ZERO_ERANGE;
    const Workspace w = workspace_layout(rows, hidden);
    if (zero_status s = check_workspace_bytes(workspace, workspace_bytes, w.bytes))
        return s;
    const Span in[] = {matrix(d_out, rows, hidden, row_stride, esize(dtype)), vec(tokens, rows, 8)};
    const Span to[] = {matrix(d_table, vocab, hidden, table_stride, esize(table_dtype)),
                       {w.bytes ? workspace : nullptr, w.bytes, 16}};
    if (zero_status s = check_spans(in, 2, to, 2))
        return s;
    if (rows == 0 && accumulate)
        return ZERO_OK;
    EmbeddingGradArgs a{};
    a.d_out = d_out;
    a.stride = row_stride;
    a.tokens = tokens;
    a.d_table = d_table;
    a.table_stride = table_stride;
    a.rows = (int32_t)rows;
    a.vocab = (int32_t)vocab;
    a.hidden = (int32_t)hidden;
    a.dtype = dtype;
    a.table_dtype = table_dtype;
    a.accumulate = accumulate;
    a.scale = scale;
    char *base = static_cast<char *>(workspace);
    if (rows > 0) {
        a.chunk_key = reinterpret_cast<uint32_t *>(base + w.chunk_key);
        a.chunk_row = reinterpret_cast<uint32_t *>(base + w.chunk_row);
        a.samples = w.samples < 0 ? nullptr : reinterpret_cast<uint32_t *>(base + w.samples);
        a.key = reinterpret_cast<uint32_t *>(base + w.key);
        a.row = reinterpret_cast<uint32_t *>(base + w.row);
        a.parts = reinterpret_cast<float *>(base + w.parts);
    }
    a.chunk = w.chunk;
    a.segment = w.segment;
    a.segments = w.segments;
    a.columns = w.columns;
    return done(launch_embedding_grad(a, stream), "zero_embedding_grad");
}
