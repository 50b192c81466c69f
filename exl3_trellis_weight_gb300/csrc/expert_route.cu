// expert_route.cu -- which tokens go to which experts, and what the first products read:
//   logits = x R^T, p = softmax, the top_k largest of each token (of equals the first),
//   pairs of token and expert sorted by expert into tiles of rows,
//   z = (x . left) H of each pair for its gate and its up matrix.
//
// All of it is latency: a few hundred KB are read and little is computed, so the three
// kernels start while the one before them ends.  One token of 64 experts, hidden 2048, 8 picks: 8.5 us
// from the first block to the last row; 64 tokens: 16.
#include "layer.cuh"
#include "linear_rotate.cuh"

namespace exl3 {

namespace {

constexpr int kTogether = 4;               // tokens that share a reading of an expert's router row

// ---- logits: a block for an expert and four tokens, its warps share the inputs ---------
template <typename T, bool VEC> __device__ __forceinline__ void load_router(const void *r, bool wide, int64_t at, float (&v)[8]) {
    if (!wide) {
        load8<T, VEC>(reinterpret_cast<const T *>(r) + at, v);
    } else {
        const float *f = reinterpret_cast<const float *>(r) + at;
        if (VEC) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(f)), b = __ldg(reinterpret_cast<const float4 *>(f) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = f[i];
        }
    }
}

// (the whole layer with 2, 4 and 8 warps, 64 experts 2048 / 1024: one token 39.3, 39.2 and 38.9 us, 8
// tokens 98.9, 97.7 and 96.5, 128 tokens 206.7, 207.3 and 208.1)
constexpr int kLogitWarps = 4;

template <typename T, bool VEC> __global__ void __launch_bounds__(kLogitWarps * 32) logits_kernel(const ExpertLaunch a) {
    __shared__ float place[kLogitWarps][kTogether];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = (int)(blockIdx.x % (unsigned)a.E);
    const int64_t t0 = (int64_t)(blockIdx.x / (unsigned)a.E) * kTogether;
    // (behind the last token its numbers once more)
    const T *x[kTogether];
#pragma unroll
    for (int i = 0; i < kTogether; i++)
        x[i] = reinterpret_cast<const T *>(a.x) + min(t0 + i, a.T - 1) * a.x_stride;
    float sum[kTogether] = {};
#pragma unroll 2
    for (int k = (warp * 32 + lane) * 8; k < a.H; k += kLogitWarps * 256) {
        float r[8], v[kTogether][8];
        load_router<T, VEC>(a.router, a.r_dt == EXL3_F32, (int64_t)e * a.H + k, r);
#pragma unroll
        for (int i = 0; i < kTogether; i++)
            load8<T, VEC>(x[i] + k, v[i]);
#pragma unroll
        for (int i = 0; i < kTogether; i++)
#pragma unroll
            for (int m = 0; m < 8; m++)
                sum[i] = __fmaf_rn(v[i][m], r[m], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < kTogether; i++) {
#pragma unroll
        for (int d = 16; d; d >>= 1)
            sum[i] = __fadd_rn(sum[i], __shfl_xor_sync(0xffffffffu, sum[i], d));
        if (lane == 0)
            place[warp][i] = sum[i];
    }
    __syncthreads();
    if (threadIdx.x < kTogether && t0 + threadIdx.x < a.T) {
        float v = place[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kLogitWarps; w++)
            v = __fadd_rn(v, place[w][threadIdx.x]);
        a.logits[(t0 + threadIdx.x) * a.E + e] = v;
    }
}

// ---- picks and the plan: one block ------------------------------------------------------
// a float's bits, ordered as unsigned, 1 at least; any picks are valid experts, whatever the logits are
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t b = __float_as_uint(v);
    return max((b & 0x80000000u) ? ~b : b | 0x80000000u, 1u);
}

__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k); }

// (threads of the plan; a few pairs are planned by fewer, whose barriers take less.  The whole layer,
// us, 256 threads and 1024: one token's 8 pairs 39.2 and 39.2, 7 tokens' 14 33.9 and 34.2, but 64
// tokens' 128 35.1 and 31.3, 32 tokens' 256 145.1 and 141.6 - a warp picks for a token at a time -
// 512 163.5 and 156.4, 1024 221.9 and 207.2)
constexpr int kPlanThreads = 1024, kPlanFew = 256;

// shared memory behind the counts: ids and, one after the other, the warps' keys
// of the experts and their counts of them
inline size_t plan_bytes(int64_t n, int E, int threads) { return (size_t)n * 4 + (size_t)(threads / 32) * E * 4; }

// The picks of a token, by a warp: the largest keys, of equals the lowest expert; lane j has
// the j-th and its key.  No key is 0 but one that has been picked.  Up to 32 R experts stay in
// registers (in shared memory each pick took 380 cycles; counting for each expert how many
// stand before it took longer still).
struct Pick {
    int e;
    uint32_t key;
};
__device__ __forceinline__ int pick_of(uint32_t best, int at, uint32_t &most) {
    most = __reduce_max_sync(0xffffffffu, best);
    const uint32_t who = __ballot_sync(0xffffffffu, best == most);
    if (__popc(who) == 1)
        return __shfl_sync(0xffffffffu, at, __ffs(who) - 1);
    return (int)__reduce_min_sync(0xffffffffu, best == most ? (uint32_t)at : 0xFFFFu);
}
template <int R> __device__ __forceinline__ Pick picks_few(const uint32_t *keys, int E, int top_k, int lane) {
    uint32_t k[R];
#pragma unroll
    for (int i = 0; i < R; i++)
        k[i] = lane + 32 * i < E ? keys[lane + 32 * i] : 0u;
    Pick p = {0, 0u};
    for (int j = 0; j < top_k; j++) {
        uint32_t best = k[0], most;
        int at = lane;
#pragma unroll
        for (int i = 1; i < R; i++)
            if (k[i] > best)
                best = k[i], at = lane + 32 * i;
        const int e = pick_of(best, at, most);
#pragma unroll
        for (int i = 0; i < R; i++)
            if (e == lane + 32 * i)
                k[i] = 0u;
        if (lane == j)
            p = {e, most};
    }
    return p;
}
__device__ __forceinline__ Pick picks_many(uint32_t *keys, int E, int top_k, int lane) {
    Pick p = {0, 0u};
    uint32_t best = 0, most;
    int at = 0;
    auto own = [&]() {                     // (found again only where one of the lane's is picked)
        best = 0;
        for (int e = lane; e < E; e += 32) {
            const uint32_t k = keys[e];
            if (k > best)
                best = k, at = e;
        }
    };
    own();
    for (int j = 0; j < top_k; j++) {
        const int e = pick_of(best, at, most);
        if (lane == (e & 31)) {
            keys[e] = 0;
            own();
        }
        if (lane == j)
            p = {e, most};
        __syncwarp();
    }
    return p;
}

template <bool ROUTE, int THREADS> __global__ void __launch_bounds__(THREADS) plan_kernel(const ExpertLaunch a) {
    constexpr int kPlanWarps = THREADS / 32;
    __shared__ int32_t count[kMaxExperts], first[kMaxExperts];
    extern __shared__ int32_t plan_mem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = (int)(a.T * a.top_k), T = (int)a.T;
    int32_t *const ids = plan_mem;
    uint32_t *const keys = reinterpret_cast<uint32_t *>(plan_mem + n) + warp * a.E;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = tid; i < a.rows; i += THREADS)
        a.pair_of[i] = -1;
    const int tiles = (int)expert_tiles(a.T, a.top_k, a.E, a.tile_n);
    for (int i = tid; i < tiles * (a.F / 128); i += THREADS)
        a.up_done[i] = 0;
    for (int i = tid; i < tiles * (a.H / 128); i += THREADS)
        a.down_done[i] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (ROUTE) {
        for (int t = warp; t < T; t += kPlanWarps) {
            const float *logits = a.logits + (int64_t)t * a.E;
            float top = -INFINITY, sum = 0.0f;
            for (int e = lane; e < a.E; e += 32) {
                const float v = __ldcg(logits + e);
                keys[e] = order_of(v);
                top = fmaxf(top, v);
            }
#pragma unroll
            for (int d = 16; d; d >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (!a.normalize) {
                for (int e = lane; e < a.E; e += 32)
                    sum = __fadd_rn(sum, expf(__fsub_rn(__ldcg(logits + e), top)));
#pragma unroll
                for (int d = 16; d; d >>= 1)
                    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
            }
            // (a lane reads back keys that it wrote itself)
            const Pick pick = a.E <= 64 ? picks_few<2>(keys, a.E, a.top_k, lane) : picks_many(keys, a.E, a.top_k, lane);
            const int id = pick.e;
            const float p = lane < a.top_k ? expf(__fsub_rn(value_of(pick.key), top)) : 0.0f;
            if (a.normalize) {
                sum = p;
#pragma unroll
                for (int d = 16; d; d >>= 1)
                    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
            }
            if (lane < a.top_k) {
                ids[t * a.top_k + lane] = id;
                a.ids[t * a.top_k + lane] = id;
                a.weights[t * a.top_k + lane] = __fdiv_rn(p, sum);
            }
        }
    } else {
        for (int i = tid; i < n; i += THREADS) {
            const int e = a.ids[i];
            ids[i] = e >= 0 && e < a.E ? e : -1;
        }
    }
    __syncthreads();
    // a warp counts the experts of its share of the pairs, and each pair's place among them
    uint16_t *const seen = reinterpret_cast<uint16_t *>(plan_mem + n);          // [warp][E]
    constexpr int kMaxRounds = 4;                                               // 32 warps x 32 lanes x 4 pairs
    const int rounds = (n + THREADS - 1) / THREADS, shares = (n + 32 * rounds - 1) / (32 * rounds);
    for (int i = tid; i < shares * a.E; i += THREADS)
        seen[i] = 0;
    __syncthreads();
    uint16_t *const mine = seen + warp * a.E;
    int place[kMaxRounds];
#pragma unroll
    for (int i = 0; i < kMaxRounds; i++) {
        place[i] = 0;
        if (i < rounds && warp < shares) {
            const int p = (warp * rounds + i) * 32 + lane, e = p < n ? ids[p] : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            if (e >= 0)
                place[i] = mine[e] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (e >= 0 && (same >> lane) == 1u)                                 // the last of them
                mine[e] = (uint16_t)(place[i] + 1);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += THREADS) {
        int c = 0;
        for (int w0 = 0; w0 < shares; w0 += 8) {
            int k[8];
#pragma unroll
            for (int w = 0; w < 8; w++)
                k[w] = w0 + w < shares ? seen[(w0 + w) * a.E + e] : 0;
#pragma unroll
            for (int w = 0; w < 8; w++) {
                if (w0 + w < shares)
                    seen[(w0 + w) * a.E + e] = (uint16_t)c;
                c += k[w];
            }
        }
        count[e] = c;
    }
    __syncthreads();
    if (warp == 0) {
        // rows from multiples of 8 on, tiles of tile_n rows
        int row = 0, tile = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, c = e < a.E ? count[e] : 0;
            const int wide = (c + 7) & ~7, parts = (c + a.tile_n - 1) / a.tile_n;
            int rs = wide, ts = parts;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int r = __shfl_up_sync(0xffffffffu, rs, d), t = __shfl_up_sync(0xffffffffu, ts, d);
                if (lane >= d)
                    rs += r, ts += t;
            }
            if (e < a.E)
                first[e] = row + rs - wide;
            for (int i = 0; i < parts; i++)
                a.tiles[tile + ts - parts + i] = make_int4(e, row + rs - wide + i * a.tile_n, min(a.tile_n, c - i * a.tile_n), 0);
            row += __shfl_sync(0xffffffffu, rs, 31);
            tile += __shfl_sync(0xffffffffu, ts, 31);
        }
        if (lane == 0)
            *a.n_tiles = tile;
    }
    __syncthreads();
    // the pairs in their order: the same plan each time
#pragma unroll
    for (int i = 0; i < kMaxRounds; i++) {
        const int p = (warp * rounds + i) * 32 + lane;
        if (i < rounds && p < n && ids[p] >= 0)
            a.pair_of[first[ids[p]] + mine[ids[p]] + place[i]] = p;
    }
}

// ---- rotated activations: a block for a row and one of its two matrices --------------------
// (x in binary16: its rotation is kept in two parts, see layer.cuh)
template <typename TX, bool VEC> __global__ void __launch_bounds__(1024) pairs_kernel(const ExpertLaunch a, int order) {
    __shared__ float wmax[32];
    extern __shared__ __align__(16) float parts[];
    const int tid = threadIdx.x, warps = (int)(blockDim.x >> 5), lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (what follows may read the plan at once: it is complete here)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row = blockIdx.x;
    const int which = blockIdx.y;
    const int p = __ldcg(a.pair_of + row);
    if (p < 0)
        return;
    const int64_t t = p / a.top_k;
    const int e = __ldcg(a.ids + p);
    float *const part = parts + (tid >> 5) * (4 * kUnit);
    const TX *x = reinterpret_cast<const TX *>(a.x) + t * a.x_stride + tid * 16;
    const float *left = (which ? a.up.left : a.gate.left) + (size_t)e * a.H;
    const int64_t NP = act_rows(a.rows);
    float v[16], m = 0.0f;
    for (int k = 0; k + tid * 16 < a.H; k += blockDim.x * 16) {
        load16<TX, VEC>(x + k, v);
        mul16(left + k + tid * 16, v);
        m = max16(v, m);
    }
    m = block_max(m, wmax, warps);
    float up, down;
    row_scale(m, up, down);
    if (tid == 0)
        a.rscale[which][row] = down;
    const bool one = (int)blockDim.x * 16 >= a.H;       // the values are still there
    for (int k0 = 0; k0 < a.H; k0 += blockDim.x * 16) {
        const int k = k0 + tid * 16;
        const bool in = k < a.H;
        if (!one && in) {
            load16<TX, VEC>(x + k0, v);
            mul16(left + k, v);
        }
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = in ? __fmul_rn(v[i], up) : 0.0f;
        rotate_out128<kTwoParts<TX>>(v, a.image[which], order, NP, row, k, in, part, lane, NP * a.H * 2);
    }
}

template <typename... A> exl3_status start(void (*kernel)(A...), dim3 grid, unsigned block, size_t smem, bool early, cudaStream_t s, A... args) {
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_smem((const void *)kernel, smem);
        if (e != cudaSuccess)
            return cuda_check(e, "cudaFuncSetAttribute(expert routing)");
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
    cfg.numAttrs = early ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess)
        return cuda_check(e, "expert routing launch");
    note_launch();
    return cuda_check(cudaGetLastError(), "expert routing launch");
}

template <typename T> exl3_status route_t(const ExpertLaunch &p, cudaStream_t s) {
    const bool vec = ((uintptr_t)p.x & 15u) == 0 && p.x_stride % 8 == 0;
    exl3_status st;
    if (p.router) {
        const int64_t jobs = (p.T + kTogether - 1) / kTogether * p.E;          // (2^16 at most)
        const bool both = vec && ((uintptr_t)p.router & 15u) == 0;
        st = start(both ? logits_kernel<T, true> : logits_kernel<T, false>, dim3((unsigned)jobs), kLogitWarps * 32, 0, false, s, p);
        if (st != EXL3_OK)
            return st;
    }
    const bool few = p.T * p.top_k <= kPlanFew;
    const unsigned threads = few ? kPlanFew : kPlanThreads;
    st = start(p.router ? (few ? plan_kernel<true, kPlanFew> : plan_kernel<true, kPlanThreads>)
                        : (few ? plan_kernel<false, kPlanFew> : plan_kernel<false, kPlanThreads>),
               dim3(1), threads, plan_bytes(p.T * p.top_k, p.E, (int)threads), p.router != nullptr, s, p);
    if (st != EXL3_OK)
        return st;
    unsigned block = (unsigned)((p.H / 16 + 31) / 32 * 32);
    block = block > 1024 ? 1024 : block;
    return start(vec ? pairs_kernel<T, true> : pairs_kernel<T, false>, dim3((unsigned)p.rows, 2), block,
                 (size_t)(block / 32) * 4 * kUnit * sizeof(float), true, s, p,
                 few_order(p.K, p.transposed));
}

}  // namespace

exl3_status launch_expert_route(const ExpertLaunch &p, cudaStream_t s) {
    return p.dt == EXL3_BF16 ? route_t<__nv_bfloat16>(p, s) : route_t<__half>(p, s);
}

}  // namespace exl3
