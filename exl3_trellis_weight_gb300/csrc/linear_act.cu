// linear_act.cu -- rotated activations: z = (x . left) H per block of 128
// inputs, one row scale per token, written in binary16 in the order in which
// linear_product.cu and linear_few.cu load their token operand.
//
// 2 bytes read and 2 written per element, but bound by the issue of instructions:
// unpacking, scaling, seven spans and packing are 20 and more an element.  A thread
// owns 16 consecutive elements and eight threads a block of 128; four spans in
// registers, an exchange through shared memory, three more in registers.  The two
// rounds of packed binary32 additions make two elements an instruction.  4096 x 4096
// bf16: 20.5 us, 3.3 TB/s; 16384 x 2048 of 64 experts: 43 us, 3.1 TB/s.
#include "linear_rotate.cuh"

namespace exl3 {

namespace {

// Adapters' sums beside the rotation: one warp for a row of the token's adapter,
// 16 products a lane and round, four rounds of loads in flight
template <typename TX, bool VEC> __device__ __forceinline__ void shrink_rows(const PrepLaunch &a) {
    const int lane = threadIdx.x & 31;
    const int r = (blockIdx.y - 1) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (r >= a.rank)
        return;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int i = a.slots[t];
        float s = 0.0f;
        if (i >= 0 && i < a.n_adapters && r < (a.ranks ? min(max(a.ranks[i], 0), a.rank) : a.rank)) {
            const TX *x = reinterpret_cast<const TX *>(a.x) + t * a.stride + lane * 8;
            const TX *m = reinterpret_cast<const TX *>(a.M) + ((size_t)i * a.rank + r) * a.n + lane * 8;
#pragma unroll 4
            for (int k = 0; k < a.n; k += 256) {
                if (k + lane * 8 < a.n) {              // (n is a multiple of 128)
                    float v[8];
                    load8<TX, VEC>(x + k, v);
                    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(m + k));
                    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float2 f = unpack2<TX>(q[e]);
                        s = __fmaf_rn(v[2 * e], f.x, s);
                        s = __fmaf_rn(v[2 * e + 1], f.y, s);
                    }
                }
            }
#pragma unroll
            for (int d = 16; d; d >>= 1)
                s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
            s = __fmul_rn(s, a.gain[i]);
        }
        if (lane == 0)
            a.h[t * a.rank + r] = s;
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
// that stand at places 2s and 2s + 1.
constexpr int kUnit = 144;                 // floats from one block of 128 to the next: other banks
__device__ __forceinline__ void rotate_out128(float (&v)[16], const PrepLaunch &a, int64_t NP, int64_t t, int k, bool in,
                                              float *part, int lane) {
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
    if (a.order == 0) {
#pragma unroll
        for (int b = 0; b < 8; b++) {
            const float2 w = *reinterpret_cast<const float2 *>(unit + 4 * ((4 * b + (s >> 1)) ^ (b >> 1)) + 2 * (s & 1));
            v[2 * b] = w.x, v[2 * b + 1] = w.y;
        }
    } else {
        // the inputs at places 2s and 2s + 1
        const int j = s >> 1, h = s & 1;
        const int i0 = a.order == 1 ? j + 8 * h : 2 * j + 8 * h, i1 = a.order == 1 ? i0 + 4 : i0 + 1;
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
    for (int b = 0; b < 8; b++)
        *reinterpret_cast<uint32_t *>(a.image + act_offset(NP, t, k0 + 16 * b + 2 * s)) = pack2<__half>(v[2 * b], v[2 * b + 1]);
}

// grid: (blocks of neighbouring rows, 1 + adapters' rows); block: a multiple of 32
// threads, 16 inputs each.  ONE: a row fits one round of the block and stays in
// registers, `left` too while the expert stays the same, and the next row is on its way.
template <typename TX, bool VEC, bool ONE>
__global__ void __launch_bounds__(1024) prep_kernel(const PrepLaunch a) {
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ float wmax[2][32];
    extern __shared__ __align__(16) float parts[];
    const int tid = threadIdx.x, warps = (int)(blockDim.x >> 5), lane = tid & 31;
    float *const part = parts + (tid >> 5) * (4 * kUnit);
    const int64_t NP = act_rows(a.T);
    // the product kernel behind this one may start on the codes; it waits for this
    // kernel's end before it reads z.  (This kernel itself, or the first of those that it
    // runs beside, starts after everything before it, so the codes are complete.)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.y > 0) {
        shrink_rows<TX, VEC>(a);
        return;
    }
    if (a.offsets) {
        for (int i = tid; i <= a.E; i += blockDim.x)
            off[i] = a.offsets[i];
        __syncthreads();
    }
    const int64_t t_lo = a.T * blockIdx.x / gridDim.x, t_hi = a.T * (blockIdx.x + 1) / gridDim.x;
    const TX *x = reinterpret_cast<const TX *>(a.x) + tid * 16;
    const bool in0 = tid * 16 < a.n;
    uint4 raw[2];
    float lf[16];
    int e_left = -1, turn = 0;
    if (ONE && VEC && in0 && t_lo < t_hi)
        load16_raw(x + t_lo * a.stride, raw);
    for (int64_t t = t_lo; t < t_hi; t++) {
        int e = 0;
        if (a.offsets)
            e = expert_of(off, a.E, t);
        float v[16];
        float m = 0.0f;
        if (ONE) {
            if (VEC) {
                unpack16<TX>(raw, v);
                if (in0 && t + 1 < t_hi)
                    load16_raw(x + (t + 1) * a.stride, raw);
            } else if (in0) {
                load16<TX, false>(x + t * a.stride, v);
            }
        }
        if (e < 0) {                       // no expert: no product, the result row is 0
            uint16_t *y = reinterpret_cast<uint16_t *>(a.y) + t * a.y_stride;
            for (int c = tid; c < a.y_cols; c += blockDim.x)
                y[c] = 0;
            continue;
        }
        const float *left = a.left + (size_t)e * a.n;
        if (ONE) {
            if (e != e_left) {
                e_left = e;                // this thread's factors
                if (in0) {
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        lf[i] = 1.0f;
                    mul16(left + tid * 16, lf);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                mul2(v[i], v[i + 1], lf[i], lf[i + 1]);
            if (in0)
                m = max16(v, m);
        } else {
            for (int k = 0; k + tid * 16 < a.n; k += blockDim.x * 16) {
                load16<TX, VEC>(x + t * a.stride + k, v);
                mul16(left + k + tid * 16, v);
                m = max16(v, m);
            }
        }
        // (two places in turn: a row's reads are done before the barrier of the next)
        m = block_max(m, wmax[turn], warps);
        turn ^= 1;
        float up, down;
        row_scale(m, up, down);
        if (tid == 0)
            a.rscale[t] = down;
        for (int k0 = 0; k0 < a.n; k0 += blockDim.x * 16) {
            const int k = k0 + tid * 16;
            const bool in = k < a.n;
            if (!ONE && in) {
                load16<TX, VEC>(x + t * a.stride + k0, v);
                mul16(left + k, v);
            }
            if (!in) {
#pragma unroll
                for (int i = 0; i < 16; i++)
                    v[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                mul2(v[i], v[i + 1], up, up);
            rotate_out128(v, a, NP, t, k, in, part, lane);
        }
    }
    // what follows waits for this kernel only: it may not end before those it runs beside.
    // One block, the last to start, is enough and keeps no other from its place.
    if (blockIdx.x == gridDim.x - 1)
        asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename TX, bool VEC, bool ONE>
exl3_status launch_prep_t(const PrepLaunch &p, dim3 grid, unsigned block, cudaStream_t s) {
    const size_t smem = (size_t)(block / 32) * 4 * kUnit * sizeof(float);
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_smem((const void *)prep_kernel<TX, VEC, ONE>, smem);
        if (e != cudaSuccess)
            return cuda_check(e, "cudaFuncSetAttribute(activation rotation)");
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.beside ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, prep_kernel<TX, VEC, ONE>, p);
    if (e != cudaSuccess)
        return cuda_check(e, "activation rotation launch");
    note_launch();
    return cuda_check(cudaGetLastError(), "activation rotation launch");
}
template <typename TX> exl3_status launch_prep_x(const PrepLaunch &p, dim3 grid, unsigned block, bool vec, bool one, cudaStream_t s) {
    if (vec)
        return one ? launch_prep_t<TX, true, true>(p, grid, block, s) : launch_prep_t<TX, true, false>(p, grid, block, s);
    return one ? launch_prep_t<TX, false, true>(p, grid, block, s) : launch_prep_t<TX, false, false>(p, grid, block, s);
}

}  // namespace

exl3_status launch_prep(const PrepLaunch &p, cudaStream_t s) {
    const bool vec = ((uintptr_t)p.x & 15u) == 0 && p.stride % 8 == 0;
    unsigned block = (unsigned)((p.n / 16 + 31) / 32 * 32);
    block = block > 1024 ? 1024 : block;
    const bool one = (int64_t)block * 16 >= p.n;
    const int64_t most = (int64_t)device_sm_count() * (1024 / block);
    const dim3 grid((unsigned)(p.T < most ? p.T : most),
                    1 + (p.n_adapters ? (unsigned)((p.rank + block / 32 - 1) / (block / 32)) : 0u));
    return p.dt == EXL3_BF16 ? launch_prep_x<__nv_bfloat16>(p, grid, block, vec, one, s)
                             : launch_prep_x<__half>(p, grid, block, vec, one, s);
}

}  // namespace exl3
