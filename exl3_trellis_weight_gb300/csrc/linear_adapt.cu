// linear_adapt.cu -- low-rank adapters of many requests: the products with the
// rank-sized side (shrink) and the sums of outer products that are their
// gradients (outer).  Simple form.
#include "linear.cuh"

namespace exl3 {

namespace {

__device__ __forceinline__ int rank_of(const int32_t *ranks, int i, int rank) {
    return ranks ? min(max(ranks[i], 0), rank) : rank;
}

// grid (T, ceil(rank / 8)): one warp per row of the token's adapter
template <typename TX>
__global__ void __launch_bounds__(256) shrink_kernel(const ShrinkLaunch a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t t = blockIdx.x;
    const int j = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (j >= a.rank)
        return;
    const int i = a.slots[t];
    float s = 0.0f;
    if (i >= 0 && i < a.n_adapters && j < rank_of(a.ranks, i, a.rank)) {
        const TX *x = reinterpret_cast<const TX *>(a.x) + t * a.stride;
        const TX *m = reinterpret_cast<const TX *>(a.M) + ((size_t)i * a.rank + j) * a.n;
        for (int k = lane; k < a.n; k += 32)
            s = __fmaf_rn(to_f32(x[k]), to_f32(m[k]), s);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
        s = __fmul_rn(s, a.gain[i]);
    }
    if (lane == 0)
        a.h[t * a.rank + j] = s;
}

// grid (n / 128, rank, n_adapters)
template <typename TX>
__global__ void __launch_bounds__(128) outer_kernel(const OuterLaunch a) {
    const int k = blockIdx.x * 128 + threadIdx.x, j = blockIdx.y, i = blockIdx.z;
    float s = 0.0f;
    if (j < rank_of(a.ranks, i, a.rank))
        for (int64_t t = 0; t < a.T; t++)
            if (a.slots[t] == i)
                s = __fmaf_rn(a.h[t * a.rank + j], to_f32(reinterpret_cast<const TX *>(a.x)[t * a.stride + k]), s);
    reinterpret_cast<TX *>(a.dM)[((size_t)i * a.rank + j) * a.n + k] = from_f32<TX>(s);
}

}  // namespace

exl3_status launch_shrink(const ShrinkLaunch &p, cudaStream_t s) {
    const dim3 grid((unsigned)p.T, (unsigned)((p.rank + 7) / 8));
    if (p.dt == EXL3_BF16)
        shrink_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    else
        shrink_kernel<__half><<<grid, 256, 0, s>>>(p);
    note_launch();
    return cuda_check(cudaGetLastError(), "adapter shrink launch");
}

exl3_status launch_outer(const OuterLaunch &p, cudaStream_t s) {
    const dim3 grid((unsigned)(p.n / 128), (unsigned)p.rank, (unsigned)p.n_adapters);
    if (p.dt == EXL3_BF16)
        outer_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p);
    else
        outer_kernel<__half><<<grid, 128, 0, s>>>(p);
    note_launch();
    return cuda_check(cudaGetLastError(), "adapter gradient launch");
}

}  // namespace exl3
