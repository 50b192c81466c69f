// expert_down.cu -- the last product of an expert layer and the sum over a token's experts.
//
// A block is 128 outputs of one expert's rows, its two groups of eight warps and the
// blocks of a cluster split the inputs.  The rotated inputs come in binary16 with a power
// of two for each 128; a block brings its share of a row to the largest of them on the
// way into shared memory.  A pair's part of the result goes to memory in binary32, and
// whoever finishes the last pair of a token adds them up in the order of the picks.
#include "expert_few.cuh"

namespace exl3 {

namespace {

using namespace tc;

struct DownArgs {
    ExpertMatrix m;
    const unsigned char *inner;
    const float *inner_scale;
    const int4 *tiles;
    const int32_t *n_tiles;
    const int32_t *pair_of, *valid;
    const int32_t *ids;
    const float *weights;
    int E, top_k;
    int64_t rows;
    int H, F;
    float *part;
    int32_t *done;
    void *y;
    int dt;
    int64_t y_stride;
    int split;
    uint32_t ring_off;
};

template <int K, bool TR, int NB>
__global__ void __launch_bounds__(kExpertThreads, 2) down_kernel(const __grid_constant__ DownArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(16) float right[128];
    __shared__ float rscale[NB * 8];
    const uint32_t base = (saddr(smem_raw) + 1023u) & ~1023u;
    unsigned char *const sb = smem_raw + (base - saddr(smem_raw));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)(blockIdx.x % a.split);
    const int nf = a.H / 128;
    const int it = (int)(blockIdx.x / a.split), tile = it / nf, f0 = it % nf * 128;
    // (the plan is complete: the launches before this one waited for it)
    if (tile >= __ldcg(a.n_tiles)) {                          // the same in all blocks of the cluster
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int4 tl = __ldcg(a.tiles + tile);
    const int e = tl.x, row0 = tl.y, n = tl.z, rows_z = (n + 7) / 8 * 8;
    const int steps = a.F / 128;
    const int k_lo = steps * rank / a.split * 2, k_hi = steps * (rank + 1) / a.split * 2;
    const int fw = warp & 7, slice = warp >> 3;
    const int q_lo = (k_hi - k_lo) * slice / 2 * 4, q_hi = (k_hi - k_lo) * (slice + 1) / 2 * 4;
    const int64_t NP = act_rows(a.rows);
    const int64_t tiles_c = (TR ? a.F : a.H) / 16, tiles_r = (TR ? a.H : a.F) / 16;
    const int64_t hop = (TR ? 1 : tiles_c) * (32 * K);
    const int64_t first = (int64_t)e * tiles_r * tiles_c +
                          (TR ? (int64_t)(f0 / 16 + fw) * tiles_c + k_lo * 4 : (int64_t)k_lo * 4 * tiles_c + f0 / 16 + fw);
    const CodeRing<K> ring(base + a.ring_off + (uint32_t)warp * CodeRing<K>::kBytes,
                           reinterpret_cast<const char *>(a.m.codes) + first * (32 * K), hop, q_lo, q_hi, lane);
    ring.begin();
    if (tid < 128)
        right[tid] = __fmul_rn(__ldg(a.m.right + (size_t)e * a.H + f0 + tid), __fmul_rn(__ldg(a.m.scale + e), 0x1p-7f));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the largest scale of a row's share
    if (tid < NB * 8) {
        float m = 0.0f;
        if (tid < n)
            for (int k = k_lo / 2; k < k_hi / 2; k++)
                m = fmaxf(m, __ldcg(a.inner_scale + (int64_t)(row0 + tid) * steps + k));
        rscale[tid] = m;
    }
    __syncthreads();
    for (int c = tid; c < (k_hi - k_lo) * rows_z * 8; c += kExpertThreads) {
        const int chunk = c & 7, r = (c >> 3) % rows_z, k = (c >> 3) / rows_z;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (r < n) {
            w = __ldcg(reinterpret_cast<const uint4 *>(a.inner + ((int64_t)(k_lo + k) * NP + row0 + r) * 128 + chunk * 16));
            // powers of two: at most 1, below 2^-24 the block is nothing beside the row's largest
            const float f = __fdiv_rn(__ldcg(a.inner_scale + (int64_t)(row0 + r) * steps + (k_lo + k) / 2), rscale[r]);
            const __half2 h = __float2half2_rn(f);
            __half2 *v = reinterpret_cast<__half2 *>(&w);
#pragma unroll
            for (int i = 0; i < 4; i++)
                v[i] = __hmul2(v[i], h);
        }
        *reinterpret_cast<uint4 *>(sb + (uint32_t)k * (NB * 1024u) + (uint32_t)r * 128u + (uint32_t)chunk * 16u) = w;
    }
    __syncthreads();
    float acc[NB][4];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            acc[b][i] = 0.0f;
    few_sums<K, TR, NB>(ring, base, rows_z / 8, lane, acc);
    __syncthreads();                       // the activations are read
    put_sums<K, TR, NB>(reinterpret_cast<float *>(sb) + slice * (NB * 8 * 128), acc, fw, lane, rscale);
    if (a.split > 1)
        cluster_sync();
    else
        __syncthreads();

    // a warp takes four rows at a time: eight lanes a row, lane u outputs 8u + 64m + i
    const int u = lane & 7;
    const int mine = (n + a.split - 1 - rank) / a.split;
    for (int i = warp * 4; i < mine; i += kExpertWarps * 4) {
        __syncwarp();                      // (rows behind the last one left the turn early)
        const int r = rank + (i + (lane >> 3)) * a.split;
        const bool in = r < n;
        float v[16];
#pragma unroll
        for (int m = 0; m < 16; m++)
            v[m] = 0.0f;
        if (in)
#pragma unroll 1
            for (int b = 0; b < a.split; b++)
#pragma unroll
                for (int s = 0; s < 2; s++)
                    add_sums(v, at_block(base + (uint32_t)((s * NB * 8 + r) * 512), b), u);
        const int p = in ? __ldcg(a.pair_of + row0 + r) : 0;
        scale_out(v, in ? __ldcg(a.weights + p) : 0.0f, right, lane);
        const int64_t t = p / a.top_k;
        if (in) {
#pragma unroll
            for (int m = 0; m < 4; m++)
                __stcg(reinterpret_cast<float4 *>(a.part + (int64_t)p * a.H + f0 + 8 * u + 4 * (m & 1) + 64 * (m >> 1)),
                       make_float4(v[4 * m], v[4 * m + 1], v[4 * m + 2], v[4 * m + 3]));
        }
        __syncwarp();
        // the last of the token's pairs to come here
        int last = 0;
        if (in && u == 0) {
            __threadfence();
            last = atomicAdd(a.done + t * nf + f0 / 128, 1) + 1 == __ldcg(a.valid + t);
            __threadfence();
        }
        last = __shfl_sync(0xffffffffu, last, lane & 24);
        if (!last)
            continue;
#pragma unroll
        for (int m = 0; m < 16; m++)
            v[m] = 0.0f;
        for (int j = 0; j < a.top_k; j++) {
            const int64_t q = t * a.top_k + j;
            const int id = __ldcg(a.ids + q);
            if (id < 0 || id >= a.E)
                continue;
#pragma unroll
            for (int m = 0; m < 4; m++) {
                const float4 w = __ldcg(reinterpret_cast<const float4 *>(a.part + q * a.H + f0 + 8 * u + 4 * (m & 1) + 64 * (m >> 1)));
                v[4 * m] = __fadd_rn(v[4 * m], w.x), v[4 * m + 1] = __fadd_rn(v[4 * m + 1], w.y);
                v[4 * m + 2] = __fadd_rn(v[4 * m + 2], w.z), v[4 * m + 3] = __fadd_rn(v[4 * m + 3], w.w);
            }
        }
        ProductLaunch o = {};
        o.y = a.y;
        o.y_stride = a.y_stride;
        if (a.dt == EXL3_BF16)
            store_out<__nv_bfloat16>(o, f0, t, v, u);
        else
            store_out<__half>(o, f0, t, v, u);
    }
    if (a.split > 1)
        cluster_sync();
}

template <int K, bool TR, int NB> exl3_status launch_down_form(const DownArgs &a, unsigned grid, uint32_t smem, cudaStream_t s) {
    cudaError_t e = allow_smem((const void *)down_kernel<K, TR, NB>, smem);
    if (e != cudaSuccess)
        return cuda_check(e, "cudaFuncSetAttribute(expert layer, down)");
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
    e = cudaLaunchKernelEx(&cfg, down_kernel<K, TR, NB>, a);
    if (e != cudaSuccess)
        return cuda_check(e, "expert layer launch (down)");
    note_launch();
    return cuda_check(cudaGetLastError(), "expert layer launch (down)");
}

template <int K, bool TR> exl3_status launch_down_n(const DownArgs &a, int tile_n, unsigned grid, uint32_t smem, cudaStream_t s) {
    return tile_n == 8    ? launch_down_form<K, TR, 1>(a, grid, smem, s)
           : tile_n == 16 ? launch_down_form<K, TR, 2>(a, grid, smem, s)
                          : launch_down_form<K, TR, 4>(a, grid, smem, s);
}
template <int K> exl3_status launch_down_t(const DownArgs &a, bool tr, int tile_n, unsigned grid, uint32_t smem, cudaStream_t s) {
    return tr ? launch_down_n<K, true>(a, tile_n, grid, smem, s) : launch_down_n<K, false>(a, tile_n, grid, smem, s);
}

}  // namespace

exl3_status launch_expert_down(const ExpertLaunch &p, cudaStream_t s) {
    DownArgs a = {};
    a.m = p.down;
    a.inner = p.inner;
    a.inner_scale = p.inner_scale;
    a.tiles = p.tiles;
    a.n_tiles = p.n_tiles;
    a.pair_of = p.pair_of;
    a.valid = p.valid;
    a.ids = p.ids;
    a.weights = p.weights;
    a.E = p.E;
    a.top_k = p.top_k;
    a.rows = p.rows;
    a.H = p.H;
    a.F = p.F;
    a.part = p.part;
    a.done = p.done;
    a.y = p.y;
    a.dt = p.dt;
    a.y_stride = p.y_stride;
    const int64_t tiles = expert_tiles(p.T, p.top_k, p.E, p.tile_n) * (p.H / 128);
    ExpertShape f;
    if (!expert_shape(f, tiles, p.F, p.tile_n, p.K_down, 1, device_sm_count()))
        return set_error(EXL3_ERR_UNSUPPORTED, "%d inner channels are too many", p.F);
    a.split = f.split;
    a.ring_off = f.ring_off;
    const unsigned grid = (unsigned)(tiles * f.split);
    switch (p.K_down) {
    case 1: return launch_down_t<1>(a, p.transposed, p.tile_n, grid, f.smem, s);
    case 2: return launch_down_t<2>(a, p.transposed, p.tile_n, grid, f.smem, s);
    case 3: return launch_down_t<3>(a, p.transposed, p.tile_n, grid, f.smem, s);
    default: return launch_down_t<4>(a, p.transposed, p.tile_n, grid, f.smem, s);
    }
}

}  // namespace exl3
