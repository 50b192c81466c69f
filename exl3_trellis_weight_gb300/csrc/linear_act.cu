// linear_act.cu -- rotated activations: z = (x . left) H per block of 128
// inputs, one row scale per token, written in binary16 in the order in which
// linear_product.cu loads its token operand.
//
// A row is scaled by a power of two before it is rotated, so that the largest
// possible element of z (128 times the row's largest product) stays below
// 2^15: binary16 then holds every element down to 2^-29 of that bound at its
// full 11 bits, whatever the range of the activations; the scale is exact and
// leaves again with the row's result.
//
// Bound by memory: 2 bytes read and 2 written per element.  A thread owns 16
// consecutive elements (four butterfly spans in registers) and eight threads a
// block of 128 (three spans by shuffles): 3 shuffles per element instead of the
// 5 of one element per lane and span.
#include "linear.cuh"

namespace exl3 {

namespace {

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

__device__ __forceinline__ float max16(const float (&v)[16], float m) {
#pragma unroll
    for (int i = 0; i < 16; i++)
        m = fmaxf(m, fabsf(v[i]));
    return m;
}

// grid: rows, one block at a time; block: a multiple of 32 threads, 16 inputs
// each.  ONE: the row fits one round of the block and stays in registers.
template <typename TX, bool VEC, bool ONE>
__global__ void act_kernel(const ActLaunch a) {
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ float wmax[32];
    const int tid = threadIdx.x;
    const int64_t NP = act_rows(a.T);
    // the product kernel behind this one may start on the codes; it waits for this
    // kernel's end before it reads z.  (This kernel itself starts after everything
    // before it, so the codes are complete.)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (a.offsets) {
        for (int i = tid; i <= a.E; i += blockDim.x)
            off[i] = a.offsets[i];
        __syncthreads();
    }
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        int e = 0;
        if (a.offsets) {
            e = expert_of(off, a.E, t);
            if (e < 0) {                 // no expert: no product, the result row is 0
                uint16_t *y = reinterpret_cast<uint16_t *>(a.y) + t * a.y_stride;
                for (int c = tid; c < a.y_cols; c += blockDim.x)
                    y[c] = 0;
                continue;
            }
        }
        const TX *x = reinterpret_cast<const TX *>(a.x) + t * a.stride;
        const float *left = a.left + (size_t)e * a.n;
        float v[16];
        float m = 0.0f;
        for (int k = tid * 16; k < a.n; k += blockDim.x * 16) {
            load16<TX, VEC>(x + k, v);
            mul16(left + k, v);
            m = max16(v, m);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        __syncthreads();                 // the previous row's reads of wmax are done
        if ((tid & 31) == 0)
            wmax[tid >> 5] = m;
        __syncthreads();
        m = 0.0f;
        for (int w = 0; w < (int)(blockDim.x >> 5); w++)
            m = fmaxf(m, wmax[w]);
        // 2^(7 - floor(log2 m)): 128 m 2^.. < 2^15; tiny rows stop at 2^107, and an
        // infinite one (its results are not numbers anyway) is left to overflow
        int ex = (int)((__float_as_uint(m) >> 23) & 255u) - 127;
        ex = ex < -100 ? -100 : ex;
        const float up = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
        if (tid == 0)
            a.rscale[t] = __uint_as_float((uint32_t)(127 + ex - 7) << 23);
        for (int k0 = 0; k0 < a.n; k0 += blockDim.x * 16) {
            const int k = k0 + tid * 16;
            const bool in = k < a.n;
            if (!ONE && in) {
                load16<TX, VEC>(x + k, v);
                mul16(left + k, v);
            }
            if (!in) {
#pragma unroll
                for (int i = 0; i < 16; i++)
                    v[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 16; i++)
                v[i] = __fmul_rn(v[i], up);
#pragma unroll
            for (int h = 1; h < 16; h <<= 1)
#pragma unroll
                for (int i = 0; i < 16; i++)
                    if ((i & h) == 0) {
                        const float p = v[i], q = v[i + h];
                        v[i] = __fadd_rn(p, q);
                        v[i + h] = __fsub_rn(p, q);
                    }
#pragma unroll
            for (int h = 1; h < 8; h <<= 1) {
                const float sg = (tid & h) ? -1.0f : 1.0f;
#pragma unroll
                for (int i = 0; i < 16; i++)
                    v[i] = __fmaf_rn(sg, v[i], __shfl_xor_sync(0xffffffffu, v[i], h));
            }
            if (in) {
                uint32_t w[8];
                if (a.order == 0) {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        w[i] = pack2<__half>(v[2 * i], v[2 * i + 1]);
                } else if (a.order == 1) {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        w[i] = pack2<__half>(v[(i >> 1) + 8 * (i & 1)], v[(i >> 1) + 8 * (i & 1) + 4]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        w[i] = pack2<__half>(v[2 * (i >> 1) + 8 * (i & 1)], v[2 * (i >> 1) + 8 * (i & 1) + 1]);
                }
                *reinterpret_cast<uint4 *>(a.image + act_offset(NP, t, k)) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(a.image + act_offset(NP, t, k + 8)) = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    }
}

template <typename TX, bool VEC>
void launch_act_t(const ActLaunch &p, unsigned grid, unsigned block, bool one, cudaStream_t s) {
    if (one)
        act_kernel<TX, VEC, true><<<grid, block, 0, s>>>(p);
    else
        act_kernel<TX, VEC, false><<<grid, block, 0, s>>>(p);
}

}  // namespace

exl3_status launch_act(const ActLaunch &p, cudaStream_t s) {
    const bool vec = ((uintptr_t)p.x & 15u) == 0 && p.stride % 8 == 0;
    unsigned block = (unsigned)((p.n / 16 + 31) / 32 * 32);
    block = block > 1024 ? 1024 : block;
    const bool one = (int64_t)block * 16 >= p.n;
    const int64_t most = (int64_t)device_sm_count() * (2048 / block);
    const unsigned grid = (unsigned)(p.T < most ? p.T : most);
    if (p.dt == EXL3_BF16)
        vec ? launch_act_t<__nv_bfloat16, true>(p, grid, block, one, s)
            : launch_act_t<__nv_bfloat16, false>(p, grid, block, one, s);
    else
        vec ? launch_act_t<__half, true>(p, grid, block, one, s) : launch_act_t<__half, false>(p, grid, block, one, s);
    note_launch();
    return cuda_check(cudaGetLastError(), "activation rotation launch");
}

}  // namespace exl3
