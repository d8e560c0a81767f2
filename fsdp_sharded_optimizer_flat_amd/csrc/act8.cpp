// act8.cpp -- the entry points of the 8-bit activation checkpoints: argument
// validation and aliasing checks.  Every check runs before any device work.
#include <hip/hip_runtime.h>

#include "act8.h"
#include "call_check.h"

namespace zero {
namespace {

// Sizes of a checkpoint; `stride` and `dtype` of the other matrix over its rows.
zero_status check_rows(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1)
        return ZERO_EINVAL;
    return rows > ZERO_MAX_LOSS_ROWS || cols > ZERO_MAX_HIDDEN ? ZERO_ERANGE : ZERO_OK;
}
int64_t blocks_of(int64_t cols) { return (cols + kActBlock - 1) / kActBlock; }

zero_status check_act(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                      const uint8_t *codes, const uint8_t *scales, Act8Args *a)
{
    if (bad_dtype(dtype))
        return ZERO_EINVAL;
    if (zero_status s = check_rows(rows, cols))
        return s;
    if (stride < cols || (rows > 0 && (!x || !codes || !scales)))
        return ZERO_EINVAL;
    if (!stride_fits(rows, stride))
        return ZERO_ERANGE;
    *a = Act8Args{const_cast<void *>(x), const_cast<uint8_t *>(codes), const_cast<uint8_t *>(scales), rows,
                  stride, (int32_t)cols, (int32_t)blocks_of(cols), dtype};
    return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status zero_act8_pack(const void *x, int32_t dtype, int64_t rows, int64_t cols,
                                      int64_t row_stride, uint8_t *codes, uint8_t *scales,
                                      void *stream)
{
    Act8Args a{};
    if (zero_status s = check_act(x, dtype, rows, cols, row_stride, codes, scales, &a))
        return s;
    const Span in[] = {matrix(x, rows, cols, row_stride, esize(dtype))};
    const Span out[] = {vec(codes, rows * cols, 1), vec(scales, rows * a.blocks, 1)};
    if (zero_status s = check_spans(in, 1, out, 2))
        return s;
    return rows == 0 ? ZERO_OK : done(launch_act8_pack(a, stream), "zero_act8_pack");
}

extern "C" zero_status zero_act8_unpack(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                        int64_t cols, void *x, int32_t dtype, int64_t row_stride,
                                        void *stream)
{
    Act8Args a{};
    if (zero_status s = check_act(x, dtype, rows, cols, row_stride, codes, scales, &a))
        return s;
    const Span in[] = {vec(codes, rows * cols, 1), vec(scales, rows * a.blocks, 1)};
    const Span out[] = {matrix(x, rows, cols, row_stride, esize(dtype))};
    if (zero_status s = check_spans(in, 2, out, 1))
        return s;
    return rows == 0 ? ZERO_OK : done(launch_act8_unpack(a, stream), "zero_act8_unpack");
}

namespace {
zero_status check_grad_sizes(int64_t rows, int64_t out_features, int64_t cols)
{
    if (zero_status s = check_rows(rows, cols))
        return s;
    if (out_features < 1)
        return ZERO_EINVAL;
    return out_features > ZERO_MAX_HIDDEN ? ZERO_ERANGE : ZERO_OK;
}
int64_t parts_bytes(const Act8Split &s, int64_t out, int64_t cols)
{
    return s.splits * s.shared(out, cols) * s.tile * s.tile * 4;
}
}  // namespace

extern "C" zero_status zero_act8_weight_grad_workspace_bytes(int64_t rows, int64_t out_features,
                                                             int64_t cols, size_t *bytes)
{
    if (!bytes)
        return ZERO_EINVAL;
    if (zero_status s = check_grad_sizes(rows, out_features, cols))
        return s;
    *bytes = (size_t)parts_bytes(act8_split(rows, out_features, cols), out_features, cols);
    return ZERO_OK;
}

extern "C" zero_status zero_act8_weight_grad(const uint16_t *d_y, int64_t rows,
                                             int64_t out_features, int64_t dy_stride,
                                             const uint8_t *codes, const uint8_t *scales,
                                             int64_t cols, void *d_w, int32_t w_dtype,
                                             int64_t w_stride, int32_t accumulate,
                                             void *workspace, size_t workspace_bytes, void *stream)
{
    if (bad_dtype(w_dtype) || (accumulate != 0 && accumulate != 1))
        return ZERO_EINVAL;
    if (zero_status s = check_grad_sizes(rows, out_features, cols))
        return s;
    if (dy_stride < out_features || w_stride < cols || !d_w || (rows > 0 && (!d_y || !codes || !scales)))
        return ZERO_EINVAL;
    if (dy_stride > 8 * (int64_t)ZERO_MAX_HIDDEN || !stride_fits(out_features, w_stride))
        return ZERO_ERANGE;
    const int64_t blocks = blocks_of(cols);
    const Act8Split split = act8_split(rows, out_features, cols);
    const int64_t need = parts_bytes(split, out_features, cols);
    if (zero_status s = check_workspace_bytes(workspace, workspace_bytes, need))
        return s;
    const Span in[] = {matrix(d_y, rows, out_features, dy_stride, 2), vec(codes, rows * cols, 1),
                       vec(scales, rows * blocks, 1)};
    const Span out[] = {matrix(d_w, out_features, cols, w_stride, esize(w_dtype)),
                        {need ? workspace : nullptr, need, 16}};
    if (zero_status s = check_spans(in, 3, out, 2))
        return s;
    if (rows == 0 && accumulate)
        return ZERO_OK;
    Act8GradArgs a{};
    a.d_y = d_y;
    a.codes = codes;
    a.scales = scales;
    a.d_w = d_w;
    a.rows = rows;
    a.dy_stride = dy_stride;
    a.w_stride = w_stride;
    a.out = (int32_t)out_features;
    a.cols = (int32_t)cols;
    a.blocks = (int32_t)blocks;
    a.w_dtype = w_dtype;
    a.accumulate = accumulate;
    a.tile = split.tile;
    a.splits = split.splits;
    a.whole = split.whole;
    a.parts = static_cast<float *>(workspace);
    return done(launch_act8_weight_grad(a, stream), "zero_act8_weight_grad");
}
