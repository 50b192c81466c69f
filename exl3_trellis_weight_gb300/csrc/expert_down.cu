// expert_down.cu -- the last product of an expert layer and the sum over a token's experts.
//
// A step is 128 outputs and 128 inputs, and a set of eight warps takes it whole.  The inputs come
// in binary16 under a power of two for each 128, so that a step's products are added to the
// others under it.  A pair's part of the result goes to memory in binary32, and a small
// kernel behind adds a token's up in the order of the picks.  (The warp that finished a
// token's last pair did that at first: the fence and the atomic that told it so stood
// in the way of the next tile: 64 tokens of 64 experts, 2048 / 1024, 8 picks, K = 2 took 70 us,
// now 54, the decode's bound is 20; one token 14.)
#include "expert_few.cuh"

namespace exl3 {

namespace {

__device__ unsigned int g_down_timeouts;

struct DownArgs {
    ExpertSteps list;
    ExpertMatrix m;
    const unsigned char *inner;
    const float *inner_scale;
    const int32_t *pair_of;
    const float *weights;
    int64_t rows;
    int H, F;
    float *part;
    bool two_parts;
};

template <int K, bool TR, int RB, bool LO> struct DownOp {
    const DownArgs &a;
    int64_t hop, hop_f;       // bytes from tile to tile of codes along the inputs and the outputs
    __device__ __forceinline__ explicit DownOp(const DownArgs &a_) : a(a_) {
        const int64_t row = (int64_t)((TR ? a.F : a.H) / 16) * (32 * K);
        hop = TR ? 32 * K : row;
        hop_f = TR ? row : 32 * K;
    }
    __device__ __forceinline__ const char *codes(int, int e, int f0) const {
        return reinterpret_cast<const char *>(a.m.codes) + (int64_t)e * (a.H / 16) * (a.F / 16) * (32 * K) + f0 / 16 * hop_f;
    }
    __device__ __forceinline__ uint32_t bytes(int rows) const { return (LO ? 4u : 2u) * (uint32_t)rows * 128u + (uint32_t)rows * 4u; }
    __device__ __forceinline__ void load(uint32_t to, uint32_t bar, int row0, int k, int rows, int lane) const {
        constexpr int kCopies = LO ? 4 : 2;
        if (lane < kCopies) {              // 64 inputs of the step, and the part
            const int64_t NP = act_rows(a.rows);
            const int q = lane & 1, part = lane >> 1;
            tc::bulk_load(to + (uint32_t)(q * (LO ? 2 : 1) + part) * (RB * 1024u),
                          a.inner + part * (NP * a.F * 2) + ((int64_t)(2 * k + q) * NP + row0) * 128, (uint32_t)rows * 128u, bar);
        } else if (lane == kCopies) {      // and the rows' scales of it
            tc::bulk_load(to + kCopies * (RB * 1024u), a.inner_scale + (int64_t)k * a.rows + row0, (uint32_t)rows * 4u, bar);
        }
    }
    // right 2^-7 s, the rows' pairs (as bits) and weights
    __device__ __forceinline__ float fetch(int tid, int e, int row0, int rows, int f0) const {
        if (tid < 128)
            return __fmul_rn(__ldg(a.m.right + (size_t)e * a.H + f0 + tid), __fmul_rn(__ldg(a.m.scale + e), 0x1p-7f));
        const int r = (tid - 128) & 63;
        if (tid >= 256 || r >= rows)
            return 0.0f;
        const int p = __ldcg(a.pair_of + row0 + r);
        return tid < 192 ? __int_as_float(p) : __ldcg(a.weights + p);
    }
    __device__ __forceinline__ void finish(float4 v, const float4 &, const float *kept, int, int r, int f0, int lane) const {
        v = mul4(mul4(rotate_row(v, lane), reinterpret_cast<const float4 *>(kept)[lane]), kept[192 + r]);
        __stcg(reinterpret_cast<float4 *>(a.part + (int64_t)__float_as_int(kept[128 + r]) * a.H + f0) + lane, v);
    }
};

// ---- y_t, the sum of a token's parts: four columns a thread -------------------------------
struct SumArgs {
    const float *part;
    const int32_t *ids;
    int E, top_k, H;
    void *y;
    int64_t y_stride;
};
template <typename T> __global__ void __launch_bounds__(128) sum_kernel(const __grid_constant__ SumArgs a) {
    const int t = (int)blockIdx.x, c = (int)(blockIdx.y * 128 + threadIdx.x) * 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c >= a.H)
        return;
    float4 v = {};
    const int64_t first = (int64_t)t * a.top_k;
#pragma unroll 1
    for (int j0 = 0; j0 < a.top_k; j0 += 8) {
        // (all are asked for at once; what is no expert's is left out)
        int id[8];
        float4 u[8];
#pragma unroll
        for (int j = 0; j < 8; j++)
            id[j] = __ldcg(a.ids + first + min(j0 + j, a.top_k - 1));
#pragma unroll
        for (int j = 0; j < 8; j++)
            u[j] = __ldcg(reinterpret_cast<const float4 *>(a.part + (first + min(j0 + j, a.top_k - 1)) * a.H + c));
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j0 + j < a.top_k && id[j] >= 0 && id[j] < a.E)
                v = add4(v, u[j]);
    }
    uint16_t *y = reinterpret_cast<uint16_t *>(a.y) + t * a.y_stride + c;
    const uint2 q = make_uint2(pack2<T>(v.x, v.y), pack2<T>(v.z, v.w));
    if ((((uintptr_t)a.y | (uintptr_t)(a.y_stride * 2)) & 7u) == 0) {
        *reinterpret_cast<uint2 *>(y) = q;
    } else {
        y[0] = (uint16_t)q.x, y[1] = (uint16_t)(q.x >> 16), y[2] = (uint16_t)q.y, y[3] = (uint16_t)(q.y >> 16);
    }
}

template <int K, bool TR, int RB, bool LO>
__global__ void __launch_bounds__(kExpertThreads, 1) down_kernel(const __grid_constant__ DownArgs a) {
    run_share<K, TR, RB, LO, false>(a.list, DownOp<K, TR, RB, LO>(a), &g_down_timeouts);
}

template <int K, bool TR, int RB, bool LO> exl3_status launch_down_form(const DownArgs &a, unsigned grid, cudaStream_t s) {
    constexpr uint32_t smem = ExpertForm<K, RB, LO, false>::kSmem;
    cudaError_t e = allow_smem((const void *)down_kernel<K, TR, RB, LO>, smem);
    if (e != cudaSuccess)
        return cuda_check(e, "cudaFuncSetAttribute(expert layer, down)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kExpertThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, down_kernel<K, TR, RB, LO>, a);
    if (e != cudaSuccess)
        return cuda_check(e, "expert layer launch (down)");
    note_launch();
    return cuda_check(cudaGetLastError(), "expert layer launch (down)");
}

template <int K, bool TR> exl3_status launch_down_n(const DownArgs &a, int tile_n, unsigned grid, cudaStream_t s) {
    if (a.two_parts)
        return tile_n == 8 ? launch_down_form<K, TR, 1, true>(a, grid, s) : launch_down_form<K, TR, 2, true>(a, grid, s);
    return tile_n == 8    ? launch_down_form<K, TR, 1, false>(a, grid, s)
           : tile_n == 16 ? launch_down_form<K, TR, 2, false>(a, grid, s)
                          : launch_down_form<K, TR, 4, false>(a, grid, s);
}
template <int K> exl3_status launch_down_t(const DownArgs &a, bool tr, int tile_n, unsigned grid, cudaStream_t s) {
    return tr ? launch_down_n<K, true>(a, tile_n, grid, s) : launch_down_n<K, false>(a, tile_n, grid, s);
}

}  // namespace

exl3_status launch_expert_down(const ExpertLaunch &p, cudaStream_t s) {
    DownArgs a = {};
    a.m = p.down;
    a.inner = p.inner;
    a.inner_scale = p.inner_scale;
    a.list = {p.tiles, p.n_tiles, (int)expert_tiles(p.T, p.top_k, p.E, p.tile_n), p.H / 128, p.F / 128, p.sums, p.down_done};
    a.pair_of = p.pair_of;
    a.weights = p.weights;
    a.rows = p.rows;
    a.H = p.H;
    a.F = p.F;
    a.part = p.part;
    a.two_parts = p.dt == EXL3_F16;
    const unsigned grid = (unsigned)expert_blocks();
    exl3_status st;
    switch (p.K_down) {
    case 1: st = launch_down_t<1>(a, p.transposed, p.tile_n, grid, s); break;
    case 2: st = launch_down_t<2>(a, p.transposed, p.tile_n, grid, s); break;
    case 3: st = launch_down_t<3>(a, p.transposed, p.tile_n, grid, s); break;
    default: st = launch_down_t<4>(a, p.transposed, p.tile_n, grid, s);
    }
    if (st != EXL3_OK)
        return st;
    const SumArgs q = {p.part, p.ids, p.E, p.top_k, p.H, p.y, p.y_stride};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.T, (unsigned)((p.H + 511) / 512));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, p.dt == EXL3_BF16 ? sum_kernel<__nv_bfloat16> : sum_kernel<__half>, q);
    if (e != cudaSuccess)
        return cuda_check(e, "expert layer launch (sum)");
    note_launch();
    return cuda_check(cudaGetLastError(), "expert layer launch (sum)");
}

exl3_status expert_down_take_wait_timeouts(unsigned int *n) {
    *n = 0;
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_down_timeouts, sizeof v);
    if (e == cudaSuccess && v != 0)
        e = cudaMemcpyToSymbol(g_down_timeouts, &zero, sizeof zero);
    if (e != cudaSuccess)
        return cuda_check(e, "wait timeout count");
    *n = v;
    return EXL3_OK;
}

}  // namespace exl3
