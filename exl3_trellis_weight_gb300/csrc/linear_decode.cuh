// linear_decode.cuh -- what the kernels that multiply by coded matrices share:
// levels of the codes, the list of token tiles, the way from sums to results.
#pragma once

#include "linear_rotate.cuh"

namespace exl3 {

// Codebook levels of two windows, fl16(fl32(n c)) with n = bytesum - 510 (the
// definition): the byte sum lands in the low bits of 2^23, one packed difference
// gives n, one packed product and one conversion round it.  The multiply, the byte
// sum and the packed operations share a pipe that starts a warp every second cycle:
// 6 of its cycles a weight, and as many instructions (packed half operations, which
// need a correction for the 24-bit c, take 7).
__device__ __forceinline__ uint32_t levels2(uint32_t s0, uint32_t s1) {
    const uint32_t a = __dp4a(s0 * kMul1Mult, 0x01010101u, 0x4B000000u);
    const uint32_t b = __dp4a(s1 * kMul1Mult, 0x01010101u, 0x4B000000u);
    uint32_t v;
    asm("{\n\t.reg .b64 x, y;\n\t.reg .f32 p, q;\n\t"
        "mov.b64 x, {%1, %2};\n\t"
        "mov.b64 y, {%3, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\t"
        "mov.b64 y, {%4, %4};\n\t"
        "mul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {p, q}, x;\n\t"
        "cvt.rn.f16x2.f32 %0, q, p;\n\t}"
        : "=r"(v) : "r"(a), "r"(b), "f"(-8389118.0f), "f"(kMul1C));
    return v;
}

// ---- tiles of outputs and tokens ----------------------------------------------
// (I: the type of token numbers, of which there are at most 2^24; the few-token kernel
// keeps 64 bits, with which the compiler spills nothing, the other one 32)
template <typename I> struct OutTile {
    int e;            // expert
    int f0;           // first output
    I t0;             // first token column, a multiple of 8 (columns before lo are not stored)
    I lo, hi;         // tokens of the expert inside the tile
};

// Shared list of token tiles: expert e has first[e + 1] - first[e] of them
struct Plan {
    int32_t off[kMaxExperts + 1];
    int32_t first[kMaxExperts + 1];
};

__device__ __forceinline__ int clamp_off(int32_t v, int64_t T) { return v < 0 ? 0 : (int64_t)v > T ? (int)T : v; }

__device__ __forceinline__ int tiles_of(int lo, int hi, int tile_n) {
    return hi > lo ? (hi - (lo & ~7) + tile_n - 1) / tile_n : 0;
}

// by all `threads` threads of a block; a barrier must follow
__device__ __forceinline__ void make_plan(Plan &plan, const int32_t *offsets, int E, int64_t T, int tile_n, int tid,
                                          int threads) {
    for (int i = tid; i <= E; i += threads)
        plan.off[i] = clamp_off(offsets[i], T);
    __syncthreads();
    if (tid >= 32)
        return;
    int at = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + tid;
        const int n = e < E ? tiles_of(plan.off[e], plan.off[e + 1], tile_n) : 0;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            sum += tid >= d ? o : 0;
        }
        if (e < E)
            plan.first[e] = at + sum - n;
        at += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (tid == 0)
        plan.first[E] = at;
}

// tile `it` of nf x (token tiles): outputs fastest, so that blocks running side by
// side share their tokens.  f0 counts in units of `width` outputs.
template <typename I>
__device__ __forceinline__ OutTile<I> out_tile(const Plan *plan, int E, I T, int tile_n, int nf, int width, int64_t it) {
    OutTile<I> t;
    int j = (int)(it / nf);
    t.f0 = (int)(it % nf) * width;
    I lo = 0, hi = T;
    t.e = 0;
    if (plan) {
        int l = 0, h = E - 1;            // last e with first[e] <= j
        while (l < h) {
            const int m = (l + h + 1) >> 1;
            if (plan->first[m] <= j)
                l = m;
            else
                h = m - 1;
        }
        t.e = l;
        j -= plan->first[l];
        lo = plan->off[l];
        hi = max(lo, (I)plan->off[l + 1]);
    }
    t.t0 = (lo & ~(I)7) + (I)j * tile_n;
    t.lo = lo > t.t0 ? lo : t.t0;
    t.hi = hi < t.t0 + tile_n ? hi : t.t0 + tile_n;
    return t;
}

// ---- from sums to results -------------------------------------------------------
// One token's results pass through shared memory as 32 float4; float4 f of a row
// sits at f ^ (f / 8 & 1), so that a warp's columns (32 consecutive outputs of one
// token) and eight threads' reads (outputs 8u + 64m + i of it, u < 8) both cover
// all banks.
__device__ __forceinline__ int out_at(int f4) { return f4 ^ ((f4 >> 3) & 1); }

template <typename TY> __device__ __forceinline__ void fma8(float *v, float h, const uint4 &w) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = unpack2<TY>(q[i]);
        v[2 * i] = __fmaf_rn(h, f.x, v[2 * i]);
        v[2 * i + 1] = __fmaf_rn(h, f.y, v[2 * i + 1]);
    }
}

// ---- the same from shared memory with many tokens: H in two passes -----------------
// 32 tokens of 32 float4; float4 f of token t sits at swz(f, t): a warp writing one
// token's 32 neighbouring outputs, and the eight lanes of each 16-byte access below,
// cover all banks.
__device__ __forceinline__ int swz(int f, int t) { return f ^ ((f >> 3) & 1) ^ ((f >> 3) & 2) ^ ((t & 1) << 2); }

// first pass, in place: thread `tid` of 128 takes token tid / 4, outputs with bits 2 and 6
// equal to tid's two: spans 1, 2, 8, 16, 32
__device__ __forceinline__ void rotate_first(float *buf, int tid) {
    const int t = tid >> 2, f0 = (tid & 1) + 16 * ((tid >> 1) & 1);
    float4 *row = reinterpret_cast<float4 *>(buf) + t * 32;
    float v[32];
#pragma unroll
    for (int b = 0; b < 8; b++) {
        const float4 f = row[swz(f0 + 2 * b, t)];
        v[4 * b] = __fadd_rn(f.x, f.y), v[4 * b + 1] = __fsub_rn(f.x, f.y);
        v[4 * b + 2] = __fadd_rn(f.z, f.w), v[4 * b + 3] = __fsub_rn(f.z, f.w);
    }
    span2<2>(v);
    span2<4>(v);
    span2<8>(v);
    span2<16>(v);
#pragma unroll
    for (int b = 0; b < 8; b++)
        row[swz(f0 + 2 * b, t)] = make_float4(v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3]);
}

// second pass: outputs 8u + 64m + i of token t (m < 2, i < 8) to v[8m + i]: spans 4 and 64,
// the row's scale and right . 2^-7 s
__device__ __forceinline__ void rotate_second(const float *buf, int t, int u, float rs, const float *right, float (&v)[16]) {
    const float4 *row = reinterpret_cast<const float4 *>(buf) + t * 32;
#pragma unroll
    for (int m = 0; m < 4; m++) {
        const float4 f = row[swz(2 * u + (m & 1) + 16 * (m >> 1), t)];
        v[4 * m] = f.x, v[4 * m + 1] = f.y, v[4 * m + 2] = f.z, v[4 * m + 3] = f.w;
    }
    span2<4>(v);
    span2<8>(v);
#pragma unroll
    for (int m = 0; m < 4; m++) {
        const float4 f = reinterpret_cast<const float4 *>(right)[2 * u + (m & 1) + 16 * (m >> 1)];
        v[4 * m] = __fmul_rn(__fmul_rn(v[4 * m], rs), f.x);
        v[4 * m + 1] = __fmul_rn(__fmul_rn(v[4 * m + 1], rs), f.y);
        v[4 * m + 2] = __fmul_rn(__fmul_rn(v[4 * m + 2], rs), f.z);
        v[4 * m + 3] = __fmul_rn(__fmul_rn(v[4 * m + 3], rs), f.w);
    }
}

// v += the adapter term of token t, outputs f0 + 8u + 64m + i (m < 2, i < 8): rows
// first, first + every, ... of the token's adapter
template <typename TY>
__device__ __forceinline__ void add_adapter(const ProductLaunch &p, int n_out, int f0, int64_t t, float (&v)[16], int u,
                                            int first, int every) {
    const int ad = p.slots[t];
    if (ad < 0 || ad >= p.n_adapters)
        return;
    const int r = p.ranks ? min(max(p.ranks[ad], 0), p.rank) : p.rank;
    const TY *b = reinterpret_cast<const TY *>(p.B) + (size_t)ad * p.rank * n_out + f0 + 8 * u;
    const float *h = p.h + (int64_t)t * p.rank;
    int j = first;
    for (; j + 3 * every < r; j += 4 * every) {            // four rows in flight
        float hj[4];
        uint4 x[4];
#pragma unroll
        for (int m = 0; m < 2; m++) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                hj[i] = h[j + i * every];
                x[i] = __ldg(reinterpret_cast<const uint4 *>(b + (size_t)(j + i * every) * n_out + 64 * m));
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
                fma8<TY>(v + 8 * m, hj[i], x[i]);
        }
    }
    for (; j < r; j += every) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(b + (size_t)j * n_out));
        const uint4 y = __ldg(reinterpret_cast<const uint4 *>(b + (size_t)j * n_out + 64));
        fma8<TY>(v, h[j], x);
        fma8<TY>(v + 8, h[j], y);
    }
}

// the token's row of the adapters' part, outputs f0 + 8u + 64m + i: float4 q (q < 4) of the
// thread's (read past L1: the kernel started before the row was written)
__device__ __forceinline__ const float4 *term_at(const ProductLaunch &p, int n_out, int f0, int64_t t, int u) {
    return reinterpret_cast<const float4 *>(p.term + t * n_out + f0 + 8 * u);
}
__device__ __forceinline__ bool has_term(const ProductLaunch &p, int64_t t) {
    const int ad = p.slots[t];
    return ad >= 0 && ad < p.n_adapters;
}
__device__ __forceinline__ void add_term(const ProductLaunch &p, int n_out, int f0, int64_t t, float (&v)[16], int u) {
    if (!has_term(p, t))
        return;
    const float4 *from = term_at(p, n_out, f0, t, u);
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const float4 f = __ldcg(from + (q & 1) + 16 * (q >> 1));
        v[4 * q] = __fadd_rn(v[4 * q], f.x), v[4 * q + 1] = __fadd_rn(v[4 * q + 1], f.y);
        v[4 * q + 2] = __fadd_rn(v[4 * q + 2], f.z), v[4 * q + 3] = __fadd_rn(v[4 * q + 3], f.w);
    }
}

// sums of a token (float4 m of the thread: outputs 8u + 64 (m / 2) + 4 (m % 2) ..) to
// results in the same places: H over the 128, the row's scale, right . 2^-7 s
__device__ __forceinline__ void scale_out(float (&v)[16], float rs, const float *right, int lane) {
    // (the places are those of rotate128 up to the order of the spans)
    rotate128(v, lane);
    const int u = lane & 7;
#pragma unroll
    for (int m = 0; m < 4; m++) {
        const float4 f = reinterpret_cast<const float4 *>(right)[2 * u + (m & 1) + 16 * (m >> 1)];
        v[4 * m] = __fmul_rn(__fmul_rn(v[4 * m], rs), f.x);
        v[4 * m + 1] = __fmul_rn(__fmul_rn(v[4 * m + 1], rs), f.y);
        v[4 * m + 2] = __fmul_rn(__fmul_rn(v[4 * m + 2], rs), f.z);
        v[4 * m + 3] = __fmul_rn(__fmul_rn(v[4 * m + 3], rs), f.w);
    }
}

// one rounding, and out
template <typename TY>
__device__ __forceinline__ void store_out(const ProductLaunch &p, int f0, int64_t t, const float (&v)[16], int u) {
    TY *y = reinterpret_cast<TY *>(p.y) + (int64_t)t * p.y_stride + f0 + 8 * u;
    const bool wide = (((uintptr_t)p.y | (uintptr_t)(p.y_stride * 2)) & 15u) == 0;
#pragma unroll
    for (int m = 0; m < 2; m++) {
        if (wide) {
            *reinterpret_cast<uint4 *>(y + 64 * m) =
                make_uint4(pack2<TY>(v[8 * m], v[8 * m + 1]), pack2<TY>(v[8 * m + 2], v[8 * m + 3]),
                           pack2<TY>(v[8 * m + 4], v[8 * m + 5]), pack2<TY>(v[8 * m + 6], v[8 * m + 7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                y[64 * m + i] = from_f32<TY>(v[8 * m + i]);
        }
    }
}

// x[4m + i] += sums[from + 16 * out_at(..)] of another block's (or this one's) shared memory
__device__ __forceinline__ void add_sums(float (&x)[16], uint32_t from, int u) {
#pragma unroll
    for (int m = 0; m < 4; m++) {
        float4 f;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                     : "r"(from + 16u * out_at(2 * u + (m & 1) + 16 * (m >> 1))));
        x[4 * m] = __fadd_rn(x[4 * m], f.x);
        x[4 * m + 1] = __fadd_rn(x[4 * m + 1], f.y);
        x[4 * m + 2] = __fadd_rn(x[4 * m + 2], f.z);
        x[4 * m + 3] = __fadd_rn(x[4 * m + 3], f.w);
    }
}

}  // namespace exl3
