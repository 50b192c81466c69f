// expert_up.cu -- silu(x G) . (x U) of each expert's rows, ready for the product with D.
//
// A step is 128 outputs and 128 inputs of both matrices: eight warps decode G, eight U, for
// the same rows, so that the two halves of an output meet in the block.  With a tile's sums
// there, a row's 128 outputs are rotated, scaled, joined and - they are a block of D's
// inputs - scaled by its factors and rotated again; they go out in binary16 under a power
// of two of their own.  64 tokens of 64 experts, 2048 / 1024, 8 picks, K = 2: 88 us at 3.0
// instructions a cycle (the decode's bound is 40); one token 18.
#include "expert_few.cuh"

namespace exl3 {

namespace {

__device__ unsigned int g_up_timeouts;

struct UpArgs {
    ExpertSteps list;
    ExpertMatrix m[2];
    const float *left;        // [E][F] of D
    const unsigned char *image[2];
    const float *rscale[2];
    int64_t rows;             // of the images
    int H, F;
    int order;                // of 16 neighbouring inputs of D's product
    unsigned char *inner;
    float *inner_scale;       // [F / 128][rows]
    bool two_parts;
};

__device__ __forceinline__ float silu(float v) { return __fdiv_rn(v, __fadd_rn(1.0f, expf(-v))); }

template <int K, bool TR, int RB, bool LO> struct UpOp {
    const UpArgs &a;
    int64_t hop, hop_f;       // bytes from tile to tile of codes along the inputs and the outputs
    __device__ __forceinline__ explicit UpOp(const UpArgs &a_) : a(a_) {
        const int64_t row = (int64_t)((TR ? a.H : a.F) / 16) * (32 * K);
        hop = TR ? 32 * K : row;
        hop_f = TR ? row : 32 * K;
    }
    __device__ __forceinline__ const char *codes(int half, int e, int f0) const {
        return reinterpret_cast<const char *>(a.m[half].codes) + (int64_t)e * (a.H / 16) * (a.F / 16) * (32 * K) + f0 / 16 * hop_f;
    }
    __device__ __forceinline__ uint32_t bytes(int rows) const { return (LO ? 8u : 4u) * (uint32_t)rows * 128u; }
    __device__ __forceinline__ void load(uint32_t to, uint32_t bar, int row0, int k, int rows, int lane) const {
        if (lane < (LO ? 8 : 4)) {         // matrix and 64 inputs of the step, and the part
            const int64_t NP = act_rows(a.rows);
            const int q = lane & 3, part = lane >> 2;
            tc::bulk_load(to + (uint32_t)(q * (LO ? 2 : 1) + part) * (RB * 1024u),
                          a.image[q >> 1] + part * (NP * a.H * 2) + ((int64_t)(2 * k + (q & 1)) * NP + row0) * 128, (uint32_t)rows * 128u, bar);
        }
    }
    // right 2^-7 s of both matrices, D's left factors, the rows' scales of both images
    __device__ __forceinline__ float fetch(int tid, int e, int row0, int rows, int f0) const {
        if (tid < 256) {
            const int w = tid >> 7;
            return __fmul_rn(__ldg(a.m[w].right + (size_t)e * a.F + f0 + (tid & 127)), __fmul_rn(__ldg(a.m[w].scale + e), 0x1p-7f));
        }
        if (tid < 384)
            return __ldg(a.left + (size_t)e * a.F + f0 + (tid & 127));
        const int w = (tid - 384) >> 6, r = (tid - 384) & 63;
        return r < rows ? __ldcg(a.rscale[w] + row0 + r) : 0.0f;
    }
    __device__ __forceinline__ void finish(float4 g, float4 v, const float *kept, int row0, int r, int f0, int lane) const {
        const float4 *factors = reinterpret_cast<const float4 *>(kept) + lane;
        const int64_t row = row0 + r, NP = act_rows(a.rows);
        g = mul4(mul4(rotate_row(g, lane), kept[384 + r]), factors[0]);
        v = mul4(mul4(rotate_row(v, lane), kept[448 + r]), factors[32]);
        g = mul4(mul4(make_float4(silu(g.x), silu(g.y), silu(g.z), silu(g.w)), v), factors[64]);
        float top = fmaxf(fmaxf(fabsf(g.x), fabsf(g.y)), fmaxf(fabsf(g.z), fabsf(g.w)));
#pragma unroll
        for (int d = 16; d; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        float up, down;
        row_scale(top, up, down);
        g = rotate_row(mul4(g, up), lane);
        if (lane == 0)
            a.inner_scale[(int64_t)(f0 / 128) * a.rows + row] = down;
        const int k = f0 + 4 * lane;
#pragma unroll
        for (int part = 0; part < (LO ? 2 : 1); part++) {
            unsigned char *const inner = a.inner + part * (NP * a.F * 2);
            const uint2 w = make_uint2(pack2<__half>(g.x, g.y), pack2<__half>(g.z, g.w));
            if (a.order == 0) {
                *reinterpret_cast<uint2 *>(inner + act_offset(NP, row, k)) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int q = (k & 15) + j;                       // of sixteen
                    const int to = a.order == 1 ? 4 * (q & 3) + (q >> 2) : 4 * ((q & 7) >> 1) + (q & 1) + 2 * (q >> 3);
                    *reinterpret_cast<uint16_t *>(inner + act_offset(NP, row, (k & ~15) + to)) = (uint16_t)((j & 2 ? w.y : w.x) >> (16 * (j & 1)));
                }
            }
            const float2 p = unpack2<__half>(w.x), q = unpack2<__half>(w.y);
            g = make_float4(__fsub_rn(g.x, p.x), __fsub_rn(g.y, p.y), __fsub_rn(g.z, q.x), __fsub_rn(g.w, q.y));
        }
    }
};

template <int K, bool TR, int RB, bool LO>
__global__ void __launch_bounds__(kExpertThreads, 1) up_kernel(const __grid_constant__ UpArgs a) {
    run_share<K, TR, RB, LO, true>(a.list, UpOp<K, TR, RB, LO>(a), &g_up_timeouts);
}

template <int K, bool TR, int RB, bool LO> exl3_status launch_up_form(const UpArgs &a, unsigned grid, cudaStream_t s) {
    constexpr uint32_t smem = ExpertForm<K, RB, LO, true>::kSmem;
    cudaError_t e = allow_smem((const void *)up_kernel<K, TR, RB, LO>, smem);
    if (e != cudaSuccess)
        return cuda_check(e, "cudaFuncSetAttribute(expert layer, up)");
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
    e = cudaLaunchKernelEx(&cfg, up_kernel<K, TR, RB, LO>, a);
    if (e != cudaSuccess)
        return cuda_check(e, "expert layer launch (up)");
    note_launch();
    return cuda_check(cudaGetLastError(), "expert layer launch (up)");
}

template <int K, bool TR> exl3_status launch_up_n(const UpArgs &a, int tile_n, unsigned grid, cudaStream_t s) {
    if (a.two_parts)
        return tile_n == 8 ? launch_up_form<K, TR, 1, true>(a, grid, s) : launch_up_form<K, TR, 2, true>(a, grid, s);
    return tile_n == 8    ? launch_up_form<K, TR, 1, false>(a, grid, s)
           : tile_n == 16 ? launch_up_form<K, TR, 2, false>(a, grid, s)
                          : launch_up_form<K, TR, 4, false>(a, grid, s);
}
template <int K> exl3_status launch_up_t(const UpArgs &a, bool tr, int tile_n, unsigned grid, cudaStream_t s) {
    return tr ? launch_up_n<K, true>(a, tile_n, grid, s) : launch_up_n<K, false>(a, tile_n, grid, s);
}

}  // namespace

exl3_status launch_expert_up(const ExpertLaunch &p, cudaStream_t s) {
    UpArgs a = {};
    a.m[0] = p.gate;
    a.m[1] = p.up;
    a.left = p.down.left;
    for (int w = 0; w < 2; w++) {
        a.image[w] = p.image[w];
        a.rscale[w] = p.rscale[w];
    }
    a.list = {p.tiles, p.n_tiles, (int)expert_tiles(p.T, p.top_k, p.E, p.tile_n), p.F / 128, p.H / 128, p.sums, p.up_done};
    a.rows = p.rows;
    a.H = p.H;
    a.F = p.F;
    a.order = few_order(p.K_down, p.transposed);
    a.inner = p.inner;
    a.inner_scale = p.inner_scale;
    a.two_parts = p.dt == EXL3_F16;
    const unsigned grid = (unsigned)expert_blocks();
    switch (p.K) {
    case 1: return launch_up_t<1>(a, p.transposed, p.tile_n, grid, s);
    case 2: return launch_up_t<2>(a, p.transposed, p.tile_n, grid, s);
    case 3: return launch_up_t<3>(a, p.transposed, p.tile_n, grid, s);
    default: return launch_up_t<4>(a, p.transposed, p.tile_n, grid, s);
    }
}

exl3_status expert_up_take_wait_timeouts(unsigned int *n) {
    *n = 0;
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_up_timeouts, sizeof v);
    if (e == cudaSuccess && v != 0)
        e = cudaMemcpyToSymbol(g_up_timeouts, &zero, sizeof zero);
    if (e != cudaSuccess)
        return cuda_check(e, "wait timeout count");
    const exl3_status st = expert_down_take_wait_timeouts(n);
    *n += v;
    return st;
}

}  // namespace exl3
