// embedding.h -- what the embedding entry points (embedding.cpp) hand to the
// kernels (embedding_kernels.hip).  Not part of the public ABI.
#pragma once

#include "zero_internal.h"

namespace zero {

struct EmbeddingArgs {
    const void *table;
    int64_t vocab, stride;
    const int64_t *tokens;
    int64_t rows;
    void *out;
    int64_t out_stride;
    int32_t hidden, dtype, out_dtype;
    float scale;
};
int launch_embedding(const EmbeddingArgs &a, void *stream);

// Tokens one workgroup sorts.
constexpr int kSortChunk = 8192;

struct EmbeddingGradArgs {
    const void *d_out;
    int64_t stride;
    const int64_t *tokens;
    void *d_table;
    int64_t table_stride;
    int32_t rows, vocab, hidden, dtype, table_dtype, accumulate;
    float scale;
    // Workspace: the tokens in ascending order with their rows (sorted in chunks,
    // then as a whole), and the partial sums of runs that segments cut:
    // segments x 2 x padded columns.
    uint32_t *chunk_key, *chunk_row, *key, *row;
    float *parts;
    int32_t segment, segments, columns;
};
int launch_embedding_grad(const EmbeddingGradArgs &a, void *stream);

// Sorted tokens that one wave adds up.
int32_t embedding_segment(int64_t rows, int64_t hidden);

}  // namespace zero
