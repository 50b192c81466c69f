// expert_up.cu -- silu(x G) . (x U) of each expert's rows, ready for the product with D.
//
// A block is 128 outputs of both matrices: eight warps decode G, eight U, for the same
// rows, so that the two halves of an output meet in the block.  The blocks of a cluster
// split the inputs.  With the sums there, a row's 128 outputs are rotated, scaled, joined
// and - they are a block of D's inputs - scaled by its factors and rotated again; they go
// out in binary16 under a power of two of their own.
#include "expert_few.cuh"

namespace exl3 {

namespace {

using namespace tc;

__device__ unsigned int g_up_timeouts;

struct UpArgs {
    ExpertMatrix m[2];
    const float *left;        // [E][F] of D
    const unsigned char *image[2];
    const float *rscale[2];
    const int4 *tiles;
    const int32_t *n_tiles;
    int64_t rows;             // of the images
    int H, F;
    int order;                // of 16 neighbouring inputs of D's product
    unsigned char *inner;
    float *inner_scale;
    int split;
    uint32_t ring_off;
};

__device__ __forceinline__ float silu(float v) { return __fdiv_rn(v, __fadd_rn(1.0f, expf(-v))); }

template <int K, bool TR, int NB>
__global__ void __launch_bounds__(kExpertThreads, 2) up_kernel(const __grid_constant__ UpArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(16) float right[2][128], left[128];
    __shared__ __align__(8) unsigned long long bar_z;
    __shared__ int gave_up;
    const uint32_t base = (saddr(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)(blockIdx.x % a.split);
    const uint32_t full = saddr(&bar_z);
    if (tid == 0) {
        bar_init(full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        gave_up = 0;
    }
    __syncthreads();
    const int nf = a.F / 128;
    const int it = (int)(blockIdx.x / a.split), tile = it / nf, f0 = it % nf * 128;
    // (the plan is complete: the launch before this one waited for it)
    if (tile >= __ldcg(a.n_tiles)) {                          // the same in all blocks of the cluster
        asm volatile("griddepcontrol.wait;" ::: "memory");    // no block ends before what this kernel follows
        return;
    }
    const int4 tl = __ldcg(a.tiles + tile);
    const int e = tl.x, row0 = tl.y, n = tl.z, rows_z = (n + 7) / 8 * 8;
    // inputs of this block in blocks of 64 (an even number)
    const int steps = a.H / 128;
    const int k_lo = steps * rank / a.split * 2, k_hi = steps * (rank + 1) / a.split * 2;
    const int fw = warp & 7, which = warp >> 3;
    const int64_t NP = act_rows(a.rows);

    const int64_t tiles_c = (TR ? a.H : a.F) / 16, tiles_r = (TR ? a.F : a.H) / 16;
    const int64_t hop = (TR ? 1 : tiles_c) * (32 * K);
    const int64_t first = (int64_t)e * tiles_r * tiles_c +
                          (TR ? (int64_t)(f0 / 16 + fw) * tiles_c + k_lo * 4 : (int64_t)k_lo * 4 * tiles_c + f0 / 16 + fw);
    const CodeRing<K> ring(base + a.ring_off + (uint32_t)warp * CodeRing<K>::kBytes,
                           reinterpret_cast<const char *>(a.m[which].codes) + first * (32 * K), hop, 0, (k_hi - k_lo) * 4, lane);
    ring.begin();
    if (tid < 256) {
        const int w = tid >> 7, f = tid & 127;
        right[w][f] = __fmul_rn(__ldg(a.m[w].right + (size_t)e * a.F + f0 + f), __fmul_rn(__ldg(a.m[w].scale + e), 0x1p-7f));
        if (w == 0)
            left[f] = __ldg(a.left + (size_t)e * a.F + f0 + f);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t z_bytes = (uint32_t)(k_hi - k_lo) * (NB * 1024u);
    if (warp == 1) {
        if (lane == 0)
            bar_expect(full, 2u * (uint32_t)(k_hi - k_lo) * (uint32_t)rows_z * 128u);
        __syncwarp();
        for (int k = k_lo + lane; k < k_hi; k += 32)
#pragma unroll
            for (int w = 0; w < 2; w++)
                bulk_load(base + w * z_bytes + (uint32_t)(k - k_lo) * (NB * 1024u), a.image[w] + ((int64_t)k * NP + row0) * 128,
                          (uint32_t)rows_z * 128u, full);
    }
    float acc[NB][4];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            acc[b][i] = 0.0f;
    if (__all_sync(0xffffffffu, bar_wait(full, 0, &gave_up, &g_up_timeouts)))
        few_sums<K, TR, NB>(ring, base + which * z_bytes, rows_z / 8, lane, acc);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                       // the activations are read
    put_sums<K, TR, NB>(reinterpret_cast<float *>(smem_raw + (base - saddr(smem_raw))) + which * (NB * 8 * 128), acc, fw, lane, nullptr);
    if (a.split > 1)
        cluster_sync();
    else
        __syncthreads();

    // a warp takes four rows at a time: eight lanes a row, lane u outputs 8u + 64m + i
    const int u = lane & 7;
    const int mine = (n + a.split - 1 - rank) / a.split;              // rows rank, rank + split, ...
    for (int i = warp * 4; i < mine; i += kExpertWarps * 4) {
        __syncwarp();                      // (rows behind the last one left the turn early)
        const int r = rank + (i + (lane >> 3)) * a.split;
        const bool in = r < n;
        const int64_t row = row0 + (in ? r : 0);
        float v[2][16];
#pragma unroll
        for (int w = 0; w < 2; w++) {
#pragma unroll
            for (int m = 0; m < 16; m++)
                v[w][m] = 0.0f;
            if (in)
#pragma unroll 1
                for (int b = 0; b < a.split; b++)
                    add_sums(v[w], at_block(base + (uint32_t)((w * NB * 8 + r) * 512), b), u);
            scale_out(v[w], in ? __ldcg(a.rscale[w] + row) : 0.0f, right[w], lane);
        }
        float top = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; m++) {
            const float4 q = reinterpret_cast<const float4 *>(left)[2 * u + (m & 1) + 16 * (m >> 1)];
            const float f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; j++)
                v[0][4 * m + j] = __fmul_rn(__fmul_rn(silu(v[0][4 * m + j]), v[1][4 * m + j]), f[j]);
        }
        top = max16(v[0], top);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        float up, down;
        row_scale(top, up, down);
#pragma unroll
        for (int j = 0; j < 16; j++)
            v[0][j] = __fmul_rn(v[0][j], up);
        rotate128(v[0], lane);
        if (!in)
            continue;
        if (u == 0)
            a.inner_scale[row * nf + f0 / 128] = down;
#pragma unroll
        for (int m = 0; m < 2; m++) {
            const int k = f0 + 8 * u + 64 * m;
            if (a.order == 0) {
                *reinterpret_cast<uint4 *>(a.inner + act_offset(NP, row, k)) =
                    make_uint4(pack2<__half>(v[0][8 * m], v[0][8 * m + 1]), pack2<__half>(v[0][8 * m + 2], v[0][8 * m + 3]),
                               pack2<__half>(v[0][8 * m + 4], v[0][8 * m + 5]), pack2<__half>(v[0][8 * m + 6], v[0][8 * m + 7]));
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int q = (k & 8) + j;                        // of sixteen
                    const int to = a.order == 1 ? 4 * (q & 3) + (q >> 2) : 4 * ((q & 7) >> 1) + (q & 1) + 2 * (q >> 3);
                    *reinterpret_cast<__half *>(a.inner + act_offset(NP, row, (k & ~15) + to)) = __float2half_rn(v[0][8 * m + j]);
                }
            }
        }
    }
    if (gave_up && warp == 1)
        bar_drain(full, 0);                // nothing may be in flight when the block ends
    if (a.split > 1)
        cluster_sync();
}

template <int K, bool TR, int NB> exl3_status launch_up_form(const UpArgs &a, unsigned grid, uint32_t smem, cudaStream_t s) {
    cudaError_t e = allow_smem((const void *)up_kernel<K, TR, NB>, smem);
    if (e != cudaSuccess)
        return cuda_check(e, "cudaFuncSetAttribute(expert layer, up)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kExpertThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, up_kernel<K, TR, NB>, a);
    if (e != cudaSuccess)
        return cuda_check(e, "expert layer launch (up)");
    note_launch();
    return cuda_check(cudaGetLastError(), "expert layer launch (up)");
}

template <int K, bool TR> exl3_status launch_up_n(const UpArgs &a, int tile_n, unsigned grid, uint32_t smem, cudaStream_t s) {
    return tile_n == 8    ? launch_up_form<K, TR, 1>(a, grid, smem, s)
           : tile_n == 16 ? launch_up_form<K, TR, 2>(a, grid, smem, s)
                          : launch_up_form<K, TR, 4>(a, grid, smem, s);
}
template <int K> exl3_status launch_up_t(const UpArgs &a, bool tr, int tile_n, unsigned grid, uint32_t smem, cudaStream_t s) {
    return tr ? launch_up_n<K, true>(a, tile_n, grid, smem, s) : launch_up_n<K, false>(a, tile_n, grid, smem, s);
}

}  // namespace

int expert_tile_n(int64_t T, int top_k, int E, int H, int F, int K, int K_down) {
    const int64_t sms = device_sm_count();
    for (int n = T <= 8 ? 8 : T <= 16 ? 16 : 32; n >= 8; n /= 2) {
        ExpertShape f;
        const int64_t tiles = expert_tiles(T, top_k, E, n);
        if (expert_shape(f, tiles * (F / 128), H, n, K, 2, sms) && expert_shape(f, tiles * (H / 128), F, n, K_down, 1, sms))
            return n;
    }
    return 0;
}

exl3_status launch_expert_up(const ExpertLaunch &p, cudaStream_t s) {
    UpArgs a = {};
    a.m[0] = p.gate;
    a.m[1] = p.up;
    a.left = p.down.left;
    for (int w = 0; w < 2; w++) {
        a.image[w] = p.image[w];
        a.rscale[w] = p.rscale[w];
    }
    a.tiles = p.tiles;
    a.n_tiles = p.n_tiles;
    a.rows = p.rows;
    a.H = p.H;
    a.F = p.F;
    a.order = few_order(p.K_down, p.transposed);
    a.inner = p.inner;
    a.inner_scale = p.inner_scale;
    const int64_t tiles = expert_tiles(p.T, p.top_k, p.E, p.tile_n) * (p.F / 128);
    ExpertShape f;
    if (!expert_shape(f, tiles, p.H, p.tile_n, p.K, 2, device_sm_count()))
        return set_error(EXL3_ERR_UNSUPPORTED, "%d hidden channels are too many", p.H);
    a.split = f.split;
    a.ring_off = f.ring_off;
    const unsigned grid = (unsigned)(tiles * f.split);
    switch (p.K) {
    case 1: return launch_up_t<1>(a, p.transposed, p.tile_n, grid, f.smem, s);
    case 2: return launch_up_t<2>(a, p.transposed, p.tile_n, grid, f.smem, s);
    case 3: return launch_up_t<3>(a, p.transposed, p.tile_n, grid, f.smem, s);
    default: return launch_up_t<4>(a, p.transposed, p.tile_n, grid, f.smem, s);
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
    *n = v;
    return EXL3_OK;
}

}  // namespace exl3
