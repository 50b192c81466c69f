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

}  // namespace exl3
