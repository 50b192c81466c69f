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
            rotate_out128(v, a.image, a.order, NP, t, k, in, part, lane);
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
