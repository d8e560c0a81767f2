// act8.h -- what the entry points of the 8-bit activation checkpoints (act8.cpp)
// hand to the kernels (act8_kernels.hip, act8_gemm_kernels.hip).  Not part of the
// public ABI.
#pragma once

#include "zero_internal.h"

namespace zero {

constexpr int kActBlock = ZERO_ACT8_BLOCK;

struct Act8Args {
    void *x;                  // read by pack, written by unpack
    uint8_t *codes, *scales;
    int64_t rows, stride;
    int32_t cols, blocks, dtype;
};
int launch_act8_pack(const Act8Args &a, void *stream);
int launch_act8_unpack(const Act8Args &a, void *stream);

struct Act8GradArgs {
    const uint16_t *d_y;
    const uint8_t *codes, *scales;
    void *d_w;
    int64_t rows, dy_stride, w_stride;
    int32_t out, cols, blocks, w_dtype, accumulate;
    int32_t tile, splits;     // d_w's tiles; workgroups that share a tile's rows
    int32_t columns;          // of the parts: cols rounded up to whole quads
    float *parts;             // splits x out x columns, where splits > 1
};
struct Act8Split {
    int32_t tile, splits;
};
Act8Split act8_split(int64_t rows, int64_t out, int64_t cols);
int launch_act8_weight_grad(const Act8GradArgs &a, void *stream);

}  // namespace zero
