// layer.cuh -- launch parameters of what stands around the coded products of a layer:
// norms and 8-bit blocks (norm.cu), products in 8 bits (linear8.cu), expert layers
// (expert_route.cu, expert_up.cu, expert_down.cu); entry points in layer_abi.cu.
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

// ---- expert layers (expert_route.cu, expert_up.cu, expert_down.cu) -------------------
// y_t = sum_j w_tj (silu(x_t G_e) . (x_t U_e)) D_e, e = ids_tj the picks of token t.
// A pair is a token and one of its picks, number t top_k + j.  Pairs are sorted by expert
// into rows, an expert's from a multiple of 8 on (rows behind its last pair hold none).
struct ExpertMatrix {
    const uint32_t *codes;     // [E][rows/16][cols/16][8 K]
    const float *left, *right; // [E][inputs], [E][outputs]
    const float *scale;        // [E]
};
struct ExpertLaunch {
    const void *x;             // [T, H]
    int dt;
    int64_t T, x_stride;
    int H, F, E, top_k;
    const void *router;        // [E, H] of type r_dt, or nullptr: ids and weights are given
    int r_dt;
    bool normalize;
    ExpertMatrix gate, up, down;
    int K, K_down, transposed;
    void *y;                   // [T, H]
    int64_t y_stride;
    // workspace
    float *logits;             // [T][E]
    int32_t *ids;              // [T top_k]
    float *weights;            // [T top_k]
    int32_t *pair_of;          // [rows]: a row's pair, or -1
    int4 *tiles;               // expert, first row and rows of each tile
    int32_t *n_tiles;
    unsigned char *image[2];   // rotated activations of the rows for gate and up (act_rows(rows) x H), parts behind each other
    float *rscale[2];          // [rows]
    unsigned char *inner;      // rotated silu(.) . (.) of the rows (act_rows(rows) x F), parts behind each other
    float *inner_scale;        // [F / 128][rows]: the powers of two of its blocks
    float *sums;               // [blocks][2][2][tile_n][128]: of tiles that blocks share
    int32_t *up_done, *down_done;      // [tiles][F / 128], [tiles][H / 128]: finished steps
    float *part;               // [T top_k][H]: a pair's part of the result
    int64_t rows;              // expert_rows(T, top_k, E)
    int tile_n;                // rows of a tile
};
inline int64_t expert_rows(int64_t T, int top_k, int E) {
    const int64_t n = T * top_k, used = n < E ? n : E;
    return (n + 7 * used + 7) / 8 * 8;
}
// tiles, at most
__host__ __device__ inline int64_t expert_tiles(int64_t T, int top_k, int E, int tile_n) {
    const int64_t n = T * top_k, used = n < E ? n : E, most = used + n / tile_n;
    return most < n ? most : n;
}
// Rotated activations are multiplied in binary16.  One rounding to its 11 bits is an eighth of
// what a result in bfloat16 loses anyway, but as much as one in binary16 does, and three of
// them (x for both matrices, the inner activations) doubled its error: for those they are
// kept in two parts, the second what the first leaves over, and multiplied twice.  The decoding
// is shared, so that costs a tenth of the time.
template <typename T> constexpr bool kTwoParts = false;
template <> constexpr bool kTwoParts<__half> = true;
// Rows of a tile, by the pairs that an expert has on average: larger tiles decode codes less often,
// and each 8 rows cost a matrix instruction for 16 x 16 of them.  64 experts 2048 / 1024, 8 picks, K = 2,
// us, 8 and 16 rows: 16 tokens 125 and 129, 32 tokens 143 and 146 (there the rule's borders are);
// 16 and 32 rows: 64 tokens 160 and 169, 128 tokens 228 and 209, 256 tokens 380 and 312.  (32 rows in
// two parts are not built: their inputs are as large as those of 64.)
inline int expert_tile_n(int64_t T, int top_k, int E, bool two_parts) {
    return T <= 8 || T * top_k <= 4 * (int64_t)E ? 8 : T <= 16 || two_parts || T * top_k <= 10 * (int64_t)E ? 16 : 32;
}
inline int64_t expert_blocks() { return device_sm_count(); }
exl3_status launch_expert_route(const ExpertLaunch &p, cudaStream_t s);
exl3_status launch_expert_up(const ExpertLaunch &p, cudaStream_t s);
exl3_status launch_expert_down(const ExpertLaunch &p, cudaStream_t s);
exl3_status expert_down_take_wait_timeouts(unsigned int *n);

// two values in e4m3, the first in the low byte; beyond 448 they become 448
__device__ __forceinline__ uint32_t pack8(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

}  // namespace exl3
