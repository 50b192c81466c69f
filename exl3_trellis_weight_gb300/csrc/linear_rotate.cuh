// linear_rotate.cuh -- (x . left) H for blocks of 128 inputs, eight threads to a block.
//
// A row is scaled by a power of two before it is rotated, so that the largest
// possible element of z (128 times the row's largest product) stays below
// 2^15: binary16 then holds every element down to 2^-29 of that bound at its
// full 11 bits, whatever the range of the activations; the scale is exact and
// leaves again with the row's result.
#pragma once

#include "linear.cuh"

namespace exl3 {

template <typename TX> __device__ __forceinline__ void load16_raw(const TX *p, uint4 (&r)[2]) {
    r[0] = __ldg(reinterpret_cast<const uint4 *>(p));
    r[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
}
template <typename TX> __device__ __forceinline__ void unpack16(const uint4 (&r)[2], float (&v)[16]) {
    const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float2 f = unpack2<TX>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

template <typename TX, bool VEC>
__device__ __forceinline__ void load16(const TX *p, float (&v)[16]) {
    if constexpr (VEC) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint4 b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 f = unpack2<TX>(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = to_f32(p[i]);
    }
}

template <typename TX, bool VEC>
__device__ __forceinline__ void load8(const TX *p, float (&v)[8]) {
    if constexpr (VEC) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = unpack2<TX>(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = to_f32(p[i]);
    }
}

__device__ __forceinline__ void mul16(const float *s, float (&v)[16]) {
    const float4 *q = reinterpret_cast<const float4 *>(s);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float4 f = __ldg(q + i);
        v[4 * i] = __fmul_rn(v[4 * i], f.x);
        v[4 * i + 1] = __fmul_rn(v[4 * i + 1], f.y);
        v[4 * i + 2] = __fmul_rn(v[4 * i + 2], f.z);
        v[4 * i + 3] = __fmul_rn(v[4 * i + 3], f.w);
    }
}

// the largest magnitude of m and 16 values (a NaN is passed over)
__device__ __forceinline__ float max16(const float (&v)[16], float m) {
#pragma unroll
    for (int i = 0; i < 16; i++)
        m = fmaxf(m, fabsf(v[i]));
    return m;
}

// Powers of two: `up` takes a row whose largest product is m below 2^8 (its rotated
// elements below 2^15), `down` takes it back.  Tiny rows stop at 2^107, and an
// infinite one (its results are not numbers anyway) is left to overflow.
__device__ __forceinline__ void row_scale(float m, float &up, float &down) {
    int ex = (int)((__float_as_uint(m) >> 23) & 255u) - 127;
    ex = ex < -100 ? -100 : ex;
    up = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
    down = __uint_as_float((uint32_t)(127 + ex - 7) << 23);
}

// ---- binary32 in pairs: each half rounds as the single operation would ----------------
__device__ __forceinline__ void add2(float &a0, float &a1, float b0, float b1, float &d0, float &d1) {
    // (a, b) -> (a + b, a - b) of two neighbours at a time
    asm("{\n\t.reg .b64 a, b, s, d;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 s, a, b;\n\t"
        "sub.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, s;\n\t"
        "mov.b64 {%2, %3}, d;\n\t}"
        : "+f"(a0), "+f"(a1), "=f"(d0), "=f"(d1) : "f"(b0), "f"(b1));
}
// butterflies of span SPAN (>= 2) over N values
template <int SPAN, int N> __device__ __forceinline__ void span2(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 2)
        if ((i & SPAN) == 0)
            add2(v[i], v[i + 1], v[i + SPAN], v[i + SPAN + 1], v[i + SPAN], v[i + SPAN + 1]);
}

__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "mul.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}
// a <- s a + b
__device__ __forceinline__ void fma2(float &a0, float &a1, float s, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, s;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "mov.b64 s, {%2, %2};\n\t"
        "fma.rn.f32x2 a, s, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1) : "f"(s), "f"(b0), "f"(b1));
}

// v: elements 16 s + i of a block of 128, s = lane % 8; v <- v H
__device__ __forceinline__ void rotate128(float (&v)[16], int lane) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float p = v[i], q = v[i + 1];
        v[i] = __fadd_rn(p, q);
        v[i + 1] = __fsub_rn(p, q);
    }
    span2<2>(v);
    span2<4>(v);
    span2<8>(v);
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
        const float sg = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 16; i += 2)
            fma2(v[i], v[i + 1], sg, __shfl_xor_sync(0xffffffffu, v[i], h), __shfl_xor_sync(0xffffffffu, v[i + 1], h));
    }
}

// the largest of the block's m, in every thread; one barrier
__device__ __forceinline__ float block_max(float m, float *place, int warps) {
#pragma unroll
    for (int d = 16; d; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0)
        place[threadIdx.x >> 5] = m;
    __syncthreads();
    m = (int)(threadIdx.x & 31) < warps ? place[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int d = 16; d; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// v: elements 16 s + i of a block of 128, s = lane % 8; writes v H in binary16.  Four
// spans in registers, three after an exchange through the warp's part of shared memory
// (shuffles, 48 a thread, made 4096 x 4096 22 us instead of 20.5): then lane s has, of each sixteen, the two
// that stand at places 2s and 2s + 1.  LO: what binary16 left of them goes to a second image,
// `lo` bytes behind the first.
constexpr int kUnit = 144;                 // floats from one block of 128 to the next: other banks
template <bool LO = false>
__device__ __forceinline__ void rotate_out128(float (&v)[16], unsigned char *image, int order, int64_t NP, int64_t t, int k,
                                              bool in, float *part, int lane, int64_t lo = 0) {
    const int s = lane & 7;
    float *const unit = part + (lane >> 3) * kUnit;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float p = v[i], q = v[i + 1];
        v[i] = __fadd_rn(p, q);
        v[i + 1] = __fsub_rn(p, q);
    }
    span2<2>(v);
    span2<4>(v);
    span2<8>(v);
    // float4 f of sixteen b at (4 b + f) ^ (b / 2): eight lanes cover all banks
#pragma unroll
    for (int f = 0; f < 4; f++)
        *reinterpret_cast<float4 *>(unit + 4 * ((4 * s + f) ^ (s >> 1))) = make_float4(v[4 * f], v[4 * f + 1], v[4 * f + 2], v[4 * f + 3]);
    __syncwarp();
    if (order == 0) {
#pragma unroll
        for (int b = 0; b < 8; b++) {
            const float2 w = *reinterpret_cast<const float2 *>(unit + 4 * ((4 * b + (s >> 1)) ^ (b >> 1)) + 2 * (s & 1));
            v[2 * b] = w.x, v[2 * b + 1] = w.y;
        }
    } else {
        // the inputs at places 2s and 2s + 1
        const int j = s >> 1, h = s & 1;
        const int i0 = order == 1 ? j + 8 * h : 2 * j + 8 * h, i1 = order == 1 ? i0 + 4 : i0 + 1;
#pragma unroll
        for (int b = 0; b < 8; b++) {
            v[2 * b] = unit[4 * ((4 * b + (i0 >> 2)) ^ (b >> 1)) + (i0 & 3)];
            v[2 * b + 1] = unit[4 * ((4 * b + (i1 >> 2)) ^ (b >> 1)) + (i1 & 3)];
        }
    }
    __syncwarp();
    span2<2>(v);
    span2<4>(v);
    span2<8>(v);
    if (!in)
        return;
    const int k0 = k & ~127;
#pragma unroll
    for (int b = 0; b < 8; b++) {
        const uint32_t w = pack2<__half>(v[2 * b], v[2 * b + 1]);
        unsigned char *const to = image + act_offset(NP, t, k0 + 16 * b + 2 * s);
        *reinterpret_cast<uint32_t *>(to) = w;
        if constexpr (LO) {
            const float2 f = unpack2<__half>(w);
            *reinterpret_cast<uint32_t *>(to + lo) = pack2<__half>(__fsub_rn(v[2 * b], f.x), __fsub_rn(v[2 * b + 1], f.y));
        }
    }
}

}  // namespace exl3
