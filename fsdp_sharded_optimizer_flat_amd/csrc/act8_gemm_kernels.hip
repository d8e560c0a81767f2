// act8_gemm_kernels.hip -- a weight's gradient from an 8-bit activation checkpoint:
// d_w[o][c] = sum_r d_y[r][o] x'[r][c] on the matrix cores.
#include "act8_device.h"

namespace zero {
namespace {

using namespace dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileO = 128, kTileC = 128, kTileR = 32;

// A workgroup of four waves per 128 x 128 tile of d_w; a wave forms 64 x 64 of it
// from 16 x 16 x 32 products, the columns as the product's rows, so that a lane
// holds four neighbouring columns.
template <typename O>
__global__ __launch_bounds__(256) void weight_grad_kernel(Act8GradArgs a)
{
    __shared__ uint16_t xs[kTileR][kTileC], ys[kTileR][kTileO];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int c0 = blockIdx.x * kTileC, o0 = blockIdx.y * kTileO;
    const int wc = wave % 2 * 64, wo = wave / 2 * 64;
    f32x4 acc[4][4] = {};   // [column tile][out tile]
    for (int64_t r0 = 0; r0 < a.rows; r0 += kTileR) {
        for (int i = tid; i < kTileR * kTileC; i += 256) {
            const int r = i / kTileC, k = i % kTileC;
            const int64_t row = r0 + r;
            const int c = c0 + k, o = o0 + k;
            float x = 0.0f;
            if (row < a.rows && c < a.cols) {
                float f[4];
                widen_codes(a.codes[row * a.cols + c],
                            scale_of(a.scales[row * a.blocks + c / kActBlock]), f);
                x = f[0];
            }
            xs[r][k] = to_bf16(x);
            ys[r][k] = row < a.rows && o < a.out ? a.d_y[row * a.dy_stride + o] : 0;
        }
        __syncthreads();
        bf16x8 x[4], y[4];
        for (int t = 0; t < 4; ++t)
            for (int j = 0; j < 8; ++j) {
                x[t][j] = __builtin_bit_cast(__bf16, xs[lane / 16 * 8 + j][wc + t * 16 + lane % 16]);
                y[t][j] = __builtin_bit_cast(__bf16, ys[lane / 16 * 8 + j][wo + t * 16 + lane % 16]);
            }
        for (int s = 0; s < 4; ++s)
            for (int t = 0; t < 4; ++t)
                acc[s][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[s], y[t], acc[s][t], 0, 0, 0);
        __syncthreads();
    }
    for (int s = 0; s < 4; ++s)
        for (int t = 0; t < 4; ++t)
            for (int j = 0; j < 4; ++j) {
                const int c = c0 + wc + s * 16 + lane / 16 * 4 + j, o = o0 + wo + t * 16 + lane % 16;
                if (c < a.cols && o < a.out) {
                    O *p = static_cast<O *>(a.d_w) + (int64_t)o * a.w_stride + c;
                    *p = narrow<O>(a.accumulate ? widen<O>(*p) + acc[s][t][j] : acc[s][t][j]);
                }
            }
}

}  // namespace

int launch_act8_weight_grad(const Act8GradArgs &a, void *stream)
{
    const dim3 grid((a.cols + kTileC - 1) / kTileC, (a.out + kTileO - 1) / kTileO);
    if (a.w_dtype == ZERO_F32)
        hipLaunchKernelGGL((weight_grad_kernel<float>), grid, dim3(256), 0, reinterpret_cast<hipStream_t>(stream), a);
    else
        hipLaunchKernelGGL((weight_grad_kernel<uint16_t>), grid, dim3(256), 0, reinterpret_cast<hipStream_t>(stream),
                           a);
    return hipGetLastError();
}

}  // namespace zero
