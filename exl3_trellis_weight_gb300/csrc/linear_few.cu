// linear_few.cu -- the coded product (see linear.cuh) for few tokens: y = z V H .
// right . 2^-7 s with V decoded into registers.
//
// With few tokens the time goes into decoding, and the operand stages, barriers
// and 128-row instructions of linear_product.cu cost more than they give (a step
// of 8192 weights took 750 cycles there for 400 of decoding).  Here a warp owns 16
// outputs and a share of the inputs, and a 16 x 16 tile of codes becomes the A
// fragment of m16n8k16 instructions directly: lane (g, j) = (lane / 4, lane % 4)
// holds two outputs and four inputs.  The order of the inputs in an instruction is
// free as long as both operands have the same, and so is the order of the outputs:
// they are chosen so that the windows are cheap to cut out (struct Lane).
//
// A block is 8 warps (128 outputs) times kSlices of the inputs; the blocks of a
// cluster split the inputs further.  Codes arrive in a ring for each warp, the
// rotated activations of the block's inputs in one go (rotating them in here took
// longer, 26 against 22 us at 7 x 12288 x 4096: every block of outputs repeats it,
// while linear_act.cu overlaps this kernel's start).  Partial sums meet in shared
// memory, block r of the cluster adds up and finishes tokens r, r + split, ...; the
// adapters' terms are made before that meeting.
//
// Bound by the decode (linear_decode.cuh): 6 cycles of a quarter of an SM for 32
// weights, against 8 of its matrix pipe for 256 weights and 8 tokens.  7 x 12288 x 4096,
// K = 1: 21 us, 8 of which are that bound; the rest is the start, the activations'
// arrival and the meeting of the partial sums.
#include "linear_few.cuh"

namespace exl3 {

namespace {

using namespace tc;

constexpr int kSlices = 2;
constexpr int kWarps = 8 * kSlices, kThreadsF = kWarps * 32;
constexpr int kTok = 32;                   // tokens of a block, at most

__device__ unsigned int g_few_timeouts;

struct FewArgs {
    ProductLaunch p;
    int n_in, n_out;
    int tile_n;          // tokens of a block: 8, 16 or 32
    int split;           // blocks of a cluster
    uint32_t ring_off;   // shared memory: activations, in their place the sums later, then the rings
};

template <int K, bool TR, int NB, typename TY>
__global__ void __launch_bounds__(kThreadsF, 2) few_kernel(const __grid_constant__ FewArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ Plan plan;
    __shared__ __align__(16) float right[128];
    __shared__ __align__(8) unsigned long long bar_z;
    __shared__ int gave_up;
    const uint32_t base = (saddr(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)(blockIdx.x % a.split);
    const ProductLaunch &p = a.p;
    const uint32_t full = saddr(&bar_z);
    if (tid == 0) {
        bar_init(full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        gave_up = 0;
    }
    if (p.offsets)
        make_plan(plan, p.offsets, p.E, p.T, a.tile_n, tid, kThreadsF);
    __syncthreads();
    const int64_t n_tok = p.offsets ? plan.first[p.E] : (p.T + a.tile_n - 1) / a.tile_n;
    const int64_t it = blockIdx.x / a.split;
    const bool any = it < n_tok * (a.n_out / 128);            // the same in all blocks of the cluster
    if (!any) {
        asm volatile("griddepcontrol.wait;" ::: "memory");    // no block ends before what this kernel follows
        return;
    }
    const OutTile<int64_t> tl = out_tile<int64_t>(p.offsets ? &plan : nullptr, p.E, p.T, a.tile_n, a.n_out / 128, 128, it);
    // inputs of this block in blocks of 64 (an even number), of this warp in tiles of 16
    const int steps = a.n_in / 128;
    const int k_lo = steps * rank / a.split * 2, k_hi = steps * (rank + 1) / a.split * 2;
    const int fw = warp & 7, slice = warp >> 3;
    const int q_lo = (k_hi - k_lo) * slice / kSlices * 4, q_hi = (k_hi - k_lo) * (slice + 1) / kSlices * 4;
    const int n = (int)(tl.hi - tl.t0);                       // tokens
    const int rows_z = (n + 7) / 8 * 8;                       // token rows to load
    const int64_t NP = act_rows(p.T);

    // codes: a warp's tiles follow each other along a tile row (TR) or down a tile column
    const int64_t tiles_c = p.cols / 16;
    const int64_t hop = (TR ? 1 : tiles_c) * (32 * K);
    const int64_t first = (int64_t)tl.e * (p.rows / 16) * tiles_c +
                          (TR ? (int64_t)(tl.f0 / 16 + fw) * tiles_c + k_lo * 4 : (int64_t)k_lo * 4 * tiles_c + tl.f0 / 16 + fw);
    // a lane copies 16 bytes of one of the four tiles of a block of 64 inputs
    constexpr int kLanes = 2 * K, kAtOnce = 4;                // lanes of a tile; tiles of a copy group
    static_assert(kLanes * kAtOnce <= 32 && kTilesAhead % kAtOnce == 0, "one copy group is one instruction");
    const uint32_t ring = base + a.ring_off + (uint32_t)warp * (kTilesAhead * 32 * K);
    const char *src = reinterpret_cast<const char *>(p.codes) + first * (32 * K) + (lane / kLanes) * hop + (lane % kLanes) * 16;
    const uint32_t dst = ring + (uint32_t)lane * 16;
    auto load_tiles = [&](int q) {
        if (lane < kLanes * kAtOnce && q < q_hi)
            copy16(dst + (uint32_t)((q - q_lo) % kTilesAhead) * (32 * K), src + (int64_t)q * hop);
        copy_group();
    };
#pragma unroll
    for (int i = 0; i < kTilesAhead; i += kAtOnce)
        load_tiles(q_lo + i);

    if (warp == 0)
        for (int i = lane; i < 128; i += 32)
            right[i] = __fmul_rn(__ldg(p.right + (size_t)tl.e * a.n_out + tl.f0 + i), __fmul_rn(__ldg(p.scale + tl.e), 0x1p-7f));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");       // (the adapters' gradients)
    if (warp == 1) {
        // activations of the block's inputs: NB * 8 token rows of each block of 64
        if (lane == 0)
            bar_expect(full, (uint32_t)(k_hi - k_lo) * (uint32_t)rows_z * 128u);
        __syncwarp();
        for (int k = k_lo + lane; k < k_hi; k += 32)
            bulk_load(base + (uint32_t)(k - k_lo) * (NB * 1024u), p.image + ((int64_t)k * NP + tl.t0) * 128,
                      (uint32_t)rows_z * 128u, full);
    }
    const int g = lane >> 2, j = lane & 3;
    float acc[NB][4];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            acc[b][i] = 0.0f;
    const int blocks = rows_z / 8;         // blocks of 8 tokens that hold any
    const bool ok = __all_sync(0xffffffffu, bar_wait(full, 0, &gave_up, &g_few_timeouts));
    const Lane l = lane_of<K, TR>(g, j);
    Words tiles(ring, l);
    uint32_t left = kTilesAhead;           // tiles up to the ring's end
    // token g's four inputs of tile i: 8 bytes of chunk 2 i + j / 2 of its row
    uint32_t z = base + (uint32_t)(q_lo >> 2) * (NB * 1024u) + (uint32_t)g * 128u + ((uint32_t)((j >> 1) ^ g) << 4) +
                 (uint32_t)(j & 1) * 8u;
    for (int q = q_lo; ok && q < q_hi; q += kAtOnce, z += NB * 1024u) {
        copy_wait<kTilesAhead / kAtOnce - 1>();
        __syncwarp();
        four_tiles<K, TR, NB, 2>(tiles, l, z, blocks, acc);
        __syncwarp();                      // every lane has read the tiles that the next copies replace
        load_tiles(q + kTilesAhead);
        left -= kAtOnce;
        tiles.move(left ? kAtOnce * 32u * K : kAtOnce * 32u * K - kTilesAhead * 32u * K);
        if (left == 0)
            left = kTilesAhead;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // partial sums: [slice][token][128 outputs], float4 f of a row at out_at(f)
    __syncthreads();                       // the activations are read
    float *const sums = reinterpret_cast<float *>(smem_raw + (base - saddr(smem_raw)));
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int o = fw * 16 + (TR || K <= 2 ? g + 8 * (i >> 1) : 2 * g + (i >> 1)), t = b * 8 + 2 * j + (i & 1);
            sums[(slice * NB * 8 + t) * 128 + 4 * out_at(o >> 2) + (o & 3)] = acc[b][i];
        }
    // a warp takes four tokens at a time, with adapters one (its four groups of eight
    // lanes a quarter of the adapter's rows each, in the first round before the sums)
    const bool shared = p.B != nullptr;
    const int each = shared ? 1 : 4, sub = shared ? 0 : lane >> 3, u = lane & 7;
    const int mine = (n + a.split - 1 - rank) / a.split;
    float v[16];
    auto adapter = [&](int i) {
#pragma unroll
        for (int m = 0; m < 16; m++)
            v[m] = 0.0f;
        const int64_t t = tl.t0 + rank + i * a.split;
        if (i >= mine || t < tl.lo)
            return;
        add_adapter<TY>(p, a.n_out, tl.f0, t, v, u, lane >> 3, 4);
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 16; m++) {
            v[m] = __fadd_rn(v[m], __shfl_xor_sync(0xffffffffu, v[m], 8));
            v[m] = __fadd_rn(v[m], __shfl_xor_sync(0xffffffffu, v[m], 16));
        }
    };
    if (shared)
        adapter(warp);
    if (a.split > 1)
        cluster_sync();
    else
        __syncthreads();
    for (int i = warp * each; i < mine; i += kWarps * each) {
        const int row = rank + (i + sub) * a.split;
        const int64_t t = row < n ? tl.t0 + row : tl.hi;
        const float rs = t < tl.hi ? p.rscale[t] : 0.0f;
        if (shared && i != warp)
            adapter(i);
        float x[16];
#pragma unroll
        for (int m = 0; m < 16; m++)
            x[m] = 0.0f;
        if (row < n)
#pragma unroll 1
            for (int b = 0; b < a.split; b++) {
                const uint32_t from = at_block(base + (uint32_t)row * 512u, b);
#pragma unroll
                for (int s = 0; s < kSlices; s++)
                    add_sums(x, from + (uint32_t)(s * NB * 8 * 512), u);
            }
        scale_out(x, rs, right, lane);
        if (t >= tl.lo && t < tl.hi && (!shared || lane < 8)) {
            if (shared) {
#pragma unroll
                for (int m = 0; m < 16; m++)
                    x[m] = __fadd_rn(x[m], v[m]);
            }
            store_out<TY>(p, tl.f0, t, x, u);
        }
    }
    if (gave_up && warp == 1)
        bar_drain(full, 0);                // nothing may be in flight when the block ends
    if (a.split > 1)
        cluster_sync();
}

template <int K, bool TR, int NB, typename TY>
exl3_status launch_few_form(const FewArgs &a, unsigned grid, uint32_t smem, cudaStream_t s) {
    cudaError_t e = allow_smem((const void *)few_kernel<K, TR, NB, TY>, smem);
    if (e != cudaSuccess)
        return cuda_check(e, "cudaFuncSetAttribute(coded product, few tokens)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreadsF);
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
    e = cudaLaunchKernelEx(&cfg, few_kernel<K, TR, NB, TY>, a);
    if (e != cudaSuccess)
        return cuda_check(e, "coded product launch (few tokens)");
    note_launch();
    return cuda_check(cudaGetLastError(), "coded product launch (few tokens)");
}

template <int K, bool TR, typename TY> exl3_status launch_few_n(const FewArgs &a, unsigned grid, uint32_t smem, cudaStream_t s) {
    switch (a.tile_n) {
    case 8: return launch_few_form<K, TR, 1, TY>(a, grid, smem, s);
    case 16: return launch_few_form<K, TR, 2, TY>(a, grid, smem, s);
    default: return launch_few_form<K, TR, 4, TY>(a, grid, smem, s);
    }
}
template <int K, typename TY> exl3_status launch_few_t(const FewArgs &a, unsigned grid, uint32_t smem, cudaStream_t s) {
    return a.p.transposed ? launch_few_n<K, true, TY>(a, grid, smem, s) : launch_few_n<K, false, TY>(a, grid, smem, s);
}
template <typename TY> exl3_status launch_few_k(const FewArgs &a, unsigned grid, uint32_t smem, cudaStream_t s) {
    switch (a.p.K) {
    case 1: return launch_few_t<1, TY>(a, grid, smem, s);
    case 2: return launch_few_t<2, TY>(a, grid, smem, s);
    case 3: return launch_few_t<3, TY>(a, grid, smem, s);
    default: return launch_few_t<4, TY>(a, grid, smem, s);
    }
}

}  // namespace

int few_order(const ProductLaunch &p) { return few_order(p.K, p.transposed); }

namespace {

// Tokens of a block, blocks of a cluster and shared memory; false when there are
// too many tokens, or when the activations of a block do not fit it.
//
// Both sides, rotation and product in a replayed graph, us, this kernel / linear_product.cu:
//   4096 -> 1024, K = 2     8 tokens 10.6 / 11.9   16: 12.1 / 12.0   32: 15.1 / 13.0
//   4096 -> 4096, K = 3     8 tokens 14.4 / 14.7   16: 16.8 / 14.7   32: 32.0 / 16.6
//   4096 -> 12288, K = 4    8 tokens 27.2 / 29.5   16: 30.0 / 29.8   32: 41.2 / 30.1
//   12288 -> 4096, K = 1    8 tokens 24.6 / 26.4   16: 27.4 / 26.6   32: 60.7 / 29.3
//   64 experts 2048 -> 1024, K = 2, even    8 rows each 67.0 / 69.3   16: 70.2 / 70.9   32: 78.3 / 73.7
//     the same, skewed (largest 6 times)    8 rows each 53.8 / 54.4   16: 72.1 / 56.9   32: 108.5 / 60.8
//   16 experts, K = 3, even                 8 rows each 19.5 / 22.8   16: 20.1 / 22.9   32: 22.8 / 23.4
// So it wins up to 8 tokens, is about even at 16 and loses from 17 on, where a block has 32
// token columns: the limits, 32 tokens and 16 rows an expert, are not where the sides cross.
bool plan_few(const ProductLaunch &p, FewArgs &a, unsigned &grid, uint32_t &smem) {
    if (p.offsets ? p.T > 16 * (int64_t)p.E : p.T > kTok)
        return false;
    a.p = p;
    a.n_in = (int)(p.transposed ? p.cols : p.rows);
    a.n_out = (int)(p.transposed ? p.rows : p.cols);
    const int64_t sms = device_sm_count();
    // all tokens; experts' sizes are not known here (their tiles start at a multiple
    // of 8 and may carry up to 7 columns of others)
    const int64_t want = p.offsets ? (p.T <= 1 ? 8 : p.T <= 9 ? 16 : 32) : p.T;
    a.tile_n = want <= 8 ? 8 : want <= 16 ? 16 : 32;
    const int64_t used = p.T < p.E ? p.T : p.E;
    const int64_t tok = p.offsets ? used + (p.T + 7 * used) / a.tile_n + 1 : (p.T + a.tile_n - 1) / a.tile_n;
    const int64_t tiles = tok * (a.n_out / 128);
    // blocks that would idle share the inputs of the tiles, at least a block of 128 each
    const int steps = a.n_in / 128;
    const uint32_t sums = (uint32_t)(kSlices * a.tile_n * 512), ring = kWarps * kTilesAhead * 32u * p.K;
    auto z_bytes = [&](int split) {
        const uint32_t z = (uint32_t)((steps + split - 1) / split) * (uint32_t)a.tile_n * 256u;
        return z > sums ? z : sums;
    };
    a.split = 1;
    while (a.split < 8 && ((tiles * a.split * 2 <= 2 * sms && steps >= a.split * 2) ||
                           z_bytes(a.split) + ring > 200u * 1024u))
        a.split *= 2;
    a.ring_off = z_bytes(a.split);
    smem = a.ring_off + ring + 1024u;
    grid = (unsigned)(tiles * a.split);
    return a.ring_off + ring <= 200u * 1024u;
}

}  // namespace

bool few_eligible(const ProductLaunch &p) {
    FewArgs a;
    unsigned grid;
    uint32_t smem;
    return plan_few(p, a, grid, smem);
}

exl3_status launch_product_few(const ProductLaunch &p, cudaStream_t s) {
    FewArgs a;
    unsigned grid;
    uint32_t smem;
    if (!plan_few(p, a, grid, smem))
        return set_error(EXL3_ERR_UNSUPPORTED, "too many tokens");
    return p.dt == EXL3_BF16 ? launch_few_k<__nv_bfloat16>(a, grid, smem, s) : launch_few_k<__half>(a, grid, smem, s);
}

exl3_status few_take_wait_timeouts(unsigned int *n) {
    *n = 0;
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_few_timeouts, sizeof v);
    if (e == cudaSuccess && v != 0)
        e = cudaMemcpyToSymbol(g_few_timeouts, &zero, sizeof zero);
    if (e != cudaSuccess)
        return cuda_check(e, "wait timeout count");
    *n = v;
    return EXL3_OK;
}

}  // namespace exl3
