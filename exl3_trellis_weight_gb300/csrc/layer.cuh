// layer.cuh -- launch parameters of what stands around the coded products of a layer:
// norms and 8-bit blocks (norm.cu), products in 8 bits (linear8.cu), expert layers
// (expert_layer.cu); entry points in layer_abi.cu.
#pragma once

#include "linear.cuh"

namespace exl3 {

// A block in e4m3 whose largest magnitude is m holds codes e4m3(v inv), inv = fl(448 / m),
// and the scale fl(m / 448).  m is 2^-96 at least, so that inv is finite; an infinity or a
// NaN in a block makes its scale one, and the whole block stands for no numbers.
constexpr float kTop8 = 448.0f;
constexpr uint32_t kLeast8 = (127u - 96u) << 23;       // bits of 2^-96

constexpr int64_t kMaxNorm = 32768;                    // columns of a norm

struct NormLaunch {
    const void *x, *residual;      // [T, n], residual nullable
    int64_t x_stride, r_stride;
    int dt;
    int64_t T;
    int n;
    const void *weight;            // [n]
    int w_dt;                      // dt or EXL3_F32
    float eps;
    void *h;                       // x + residual, with residual
    int64_t h_stride;
    void *y;                       // nullable
    int64_t y_stride;
    uint8_t *y8;                   // nullable, [T][n]
    float *scale;                  // [ceil(n / 128)][T], with y8
};
exl3_status launch_norm(const NormLaunch &p, cudaStream_t s);

struct NormGradLaunch {
    const void *dy, *h, *dh;       // [T, n], dh nullable
    int64_t dy_stride, h_stride, dh_stride;
    int dt;
    int64_t T;
    int n;
    const void *weight;
    int w_dt;
    float eps;
    void *dx;
    int64_t dx_stride;
    void *dweight;                 // nullable, [n], w_dt
    float *part;                   // norm_grad_parts(T, n) * n floats, with dweight
};
// rows of partial sums of dweight
int64_t norm_grad_parts(int64_t T, int64_t n);
exl3_status launch_norm_grad(const NormGradLaunch &p, cudaStream_t s);

struct Quantize8Launch {
    const void *x;                 // [T, n]
    int dt;
    int64_t T, n, stride;
    int block_rows;                // 1 or 128
    uint8_t *codes;                // [T][n]
    float *scale;                  // 1: [ceil(n / 128)][T]; 128: [ceil(T / 128)][ceil(n / 128)]
};
exl3_status launch_quantize8(const Quantize8Launch &p, cudaStream_t s);

struct Linear8Launch {
    const uint8_t *x;              // [T, n_in] in e4m3, 16-byte aligned rows
    int64_t T, x_stride;
    const float *xs;               // scale of x's token t and block b: xs[t * xs_t + b * xs_b]
    int64_t xs_t, xs_b;
    const uint8_t *w;              // [rows, cols] in e4m3
    int64_t rows, cols;
    const float *ws;               // [ceil(rows / 128)][ceil(cols / 128)]
    int transposed;
    void *y;                       // [T, n_out]
    int dt;
    int64_t y_stride;
    bool behind;                   // x and xs are written by the launch before, the weights are not
};
exl3_status launch_linear8(const Linear8Launch &p, cudaStream_t s);

// two values in e4m3, the first in the low byte; beyond 448 they become 448
__device__ __forceinline__ uint32_t pack8(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

}  // namespace exl3
