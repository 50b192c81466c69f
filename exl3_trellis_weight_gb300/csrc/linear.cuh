// linear.cuh -- launch parameters shared by the kernels that multiply by
// trellis-coded matrices (linear_act.cu, linear_product.cu, linear_adapt.cu)
// and their entry points (linear_abi.cu).
//
// With V the codebook levels of a coded matrix, H the blockwise Sylvester
// matrix and s its scale, the decoded matrix is
//     W^ = 2^-7 s diag(su) (H V H) diag(sv),
// so a product with it needs no decoded weights in memory:
//     x W^   = ((x . su) H) V   H . sv . 2^-7 s
//     x W^^T = ((x . sv) H) V^T H . su . 2^-7 s.
// linear_act.cu makes z = (x . left) H once per token, linear_product.cu
// multiplies by V straight from the codes and rotates the result.
#pragma once

#include "common.cuh"

namespace exl3 {

constexpr int kMaxExperts = 1024;
constexpr int kMaxAdapters = 1024;
constexpr int kMaxRank = 128;

// Rotated activations z in binary16, in the order the product kernel loads
// them: for each block of 64 inputs, NP token rows of 128 bytes whose 16-byte
// chunks c sit at c ^ (row & 7) (the 128-byte swizzle of a shared-memory
// operand), so that any tile of token rows starting at a multiple of 8 is one
// contiguous copy.  NP leaves 32 rows behind the last token: tiles are rounded
// up to 16 or 32 tokens.
__host__ __device__ inline int64_t act_rows(int64_t T) { return (T + 7) / 8 * 8 + 32; }
__host__ __device__ inline int64_t act_offset(int64_t NP, int64_t t, int k) {
    return ((int64_t)(k >> 6) * NP + t) * 128 + ((((k >> 3) & 7) ^ (int)(t & 7)) << 4) + (k & 7) * 2;
}

struct PrepLaunch {
    const void *x;            // [T, n] activations, row stride in elements
    int dt;                   // EXL3_BF16 / EXL3_F16
    int64_t T, stride;
    int n;                    // inputs, a multiple of 128
    const float *left;        // [E or 1][n]
    const int32_t *offsets;   // [E + 1] or nullptr (one matrix)
    int E;
    unsigned char *image;     // act_rows(T) * n * 2 bytes
    float *rscale;            // [T]: z = image * rscale
    void *y;                  // rows outside of every expert are set to 0
    int64_t y_stride;
    int y_cols;
    // order of 16 neighbouring inputs: place 4j + i holds input 4j + i (0), j + 4i (1)
    // or 2j + i % 2 + 8 (i / 2) (2)
    int order;
    // beside it, in the same launch (n_adapters > 0):
    // h[t][r] = gain_i sum_k M[i][r][k] x[t][k], i = slots[t], r < ranks[i] (0 otherwise)
    const void *M;            // [n_adapters][rank][n]
    const float *gain;
    const int32_t *slots, *ranks;
    int n_adapters, rank;
    float *h;                 // [T][rank]
    // runs beside the kernels launched before it, which neither write what it reads nor
    // use what it writes, and ends after them (n_adapters == 0)
    bool beside;
};
exl3_status launch_prep(const PrepLaunch &p, cudaStream_t s);

struct ProductLaunch {
    const unsigned char *image;   // rotated activations (PrepLaunch)
    const float *rscale;
    int64_t T;
    const uint32_t *codes;    // [E][rows/16][cols/16][8 K]
    int64_t rows, cols;
    int K;
    const float *right;       // [E or 1][outputs]
    const float *scale;       // [E or 1]
    int transposed;
    const int32_t *offsets;   // [E + 1] or nullptr
    int E;                    // 1 when offsets == nullptr
    // adapters: B != nullptr adds sum_j h[t][j] B[slot_t][j] to the result; term != nullptr
    // adds its rows of tokens with an adapter (launch_expand)
    const void *B;            // nullable, [n_adapters][rank][outputs], dtype dt
    const float *h;           // [T][rank]
    const float *term;        // nullable, [T][outputs], 16-byte aligned
    const int32_t *slots;     // [T]
    const int32_t *ranks;     // nullable, [n_adapters]
    int n_adapters, rank;
    void *y;
    int dt;
    int64_t y_stride;
};
exl3_status launch_product(const ProductLaunch &p, cudaStream_t s);
// the same for few tokens (linear_few.cu)
bool few_eligible(const ProductLaunch &p);
int few_order(const ProductLaunch &p);     // PrepLaunch::order that it reads
exl3_status few_take_wait_timeouts(unsigned int *n);
exl3_status launch_product_few(const ProductLaunch &p, cudaStream_t s);

// Adapters of more than a few tokens (linear_adapt.cu), tokens sorted by adapter
struct AdaptPlan {
    int4 *tiles;              // adapter, first place in perm and tokens of each tile of 32
    int32_t *perm;            // [T] tokens by adapter (those without one left out)
    int32_t *seg;             // [n + 1] where an adapter's tokens begin
    int32_t *n_tiles;
    uint32_t *largest;        // [2][n]
};
size_t adapt_plan_ints(int64_t T, int n);
AdaptPlan adapt_plan(int32_t *ints, int64_t T, int n);

struct AdaptSide {
    const void *x;            // [T, n] activations
    int64_t stride;
    int n;
    const void *M;            // [n_adapters][rank][n]
    float *h;                 // [T][rank]; only rows of tokens with an adapter are written
    uint32_t *largest;        // [n_adapters] bits of the largest |h|
    void *dM;                 // like M
};
struct AdaptLaunch {
    AdaptPlan plan;
    int dt;
    int64_t T;
    int n, rank;              // adapters, and their rows
    const float *gain;
    const int32_t *slots, *ranks;
    AdaptSide side[2];
    int split;                // (set by the launchers)
};
exl3_status launch_adapt_plan(const AdaptLaunch &p, cudaStream_t s);
// sides 0 .. sides - 1: h[t] = gain_i M_i x_t
exl3_status launch_shrink(const AdaptLaunch &p, int sides, cudaStream_t s);
// term[t] = sum_r h[t][r] M_i[r] with side 0's h and M (n outputs); rows without an adapter stay
exl3_status launch_expand(const AdaptLaunch &p, float *term, cudaStream_t s);
// both sides: dM_i[r] = sum_{t of i} h[t][r] x_t
exl3_status launch_outer(const AdaptLaunch &p, cudaStream_t s);

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

// two values of a packed pair
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Expert of token t: the e with offsets[e] <= t < offsets[e + 1], or -1.
// The offsets are expected to ascend; whatever they hold, the result is a
// valid index or -1.
__device__ __forceinline__ int expert_of(const int32_t *off, int E, int64_t t) {
    int lo = 0, hi = E;                  // first e with off[e + 1] > t lies in [lo, hi]
    while (lo < hi) {
        const int m = (lo + hi) >> 1;
        if (off[m + 1] > t)
            hi = m;
        else
            lo = m + 1;
    }
    return lo < E && off[lo] <= t ? lo : -1;
}

}  // namespace exl3
