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

// Tokens one workgroup sorts: powers of two.  Sorting takes 11 us for chunks of 2048
// and 26 for 8192, putting chunks together 7 us for up to eight of them and 5 more for
// eight more, so small chunks serve up to 65536 tokens.  Small and large ones, us, tables
// cleared meanwhile: 8192 x 1280 into 50304 rows of bf16 43 and 50, 32768 x 2048 103 and
// 118, 16384 x 4096 into 128256 242 and 240; added to what is there 67 and 76.
constexpr int kSortChunk = 2048, kMaxSortChunk = 8192;
constexpr int kSamples = 128;   // of a sorted chunk's tokens, at even distances
inline int32_t embedding_chunk(int64_t rows) { return rows > 65536 ? kMaxSortChunk : kSortChunk; }

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
    uint32_t *chunk_key, *chunk_row, *samples, *key, *row;
    float *parts;
    int32_t chunk, segment, segments, columns;
};
int launch_embedding_grad(const EmbeddingGradArgs &a, void *stream);

// Sorted tokens that one wave adds up: more where rows times slabs of 512 columns exceed
// each of these.
constexpr int64_t kSegmentWork[] = {16384, 65536};
inline int64_t embedding_slabs(int64_t hidden) { return (hidden + 511) / 512; }
int32_t embedding_segment(int64_t rows, int64_t hidden);

}  // namespace zero
