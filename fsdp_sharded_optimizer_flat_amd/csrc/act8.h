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
    int32_t tile;             // d_w's tiles: tile x tile
    int32_t splits;           // workgroups that share a tile's rows, but for
    int32_t whole;            // the first tiles, which a workgroup each takes whole
    float *parts;             // splits x the other tiles x tile x tile
};
struct Act8Split {
    int32_t tile, splits, whole;
    int64_t shared(int64_t out, int64_t cols) const   // tiles that are not whole
    {
        return ((out + tile - 1) / tile) * ((cols + tile - 1) / tile) - whole;
    }
};
Act8Split act8_split(int64_t rows, int64_t out, int64_t cols);
int launch_act8_weight_grad(const Act8GradArgs &a, void *stream);

}  // namespace zero
