// linear8.cu -- y = x W (or x W^T) with both in e4m3, x with a scale for each 128 inputs of
// a token, W with one for each block of 128 x 128:
//   y[t][f] = sum over blocks b of 128 inputs of  xs[t][b] ws[b][f / 128] sum_{k in b} x8[t][k] w8[k][f]
//
// The inner sums are whole steps of the tensor cores: 128 inputs are one row of a swizzled
// operand and four instructions.  Their result leaves tensor memory after every step and is
// added up in registers in binary32 under its scale, while the next steps' products run into
// other columns of tensor memory.
//
// Two forms.  Few tokens (SWAP): the 128 rows of the instruction are outputs, tokens its
// columns, and the blocks of a cluster share the inputs of a tile; bound by reading the
// weights.  Many tokens: the rows are tokens, 128 or 256 outputs the columns, so that the
// scale is one factor of a thread's whole row; bound by the tensor cores.  A weight matrix
// is used as it lies, the operand's rows run along its inputs or along its outputs.
//
// Warps: accumulators to registers (four for each half of the columns), one that copies
// tiles, one that issues the matrix instructions, one that multiplies the scales of steps
// ahead.  (When the warps with the accumulators fetched the scales themselves, a step ahead, and
// each thread stored its row, 4096 tokens x 4096 x 12288 took 236 us; now 181 to 191, 2160 to 2280
// TFLOP/s, and 183 with W the other way round.  The tensor pipe is busy for half of the time, the issue
// slots are not the limit: the steps wait for the result warps, which take each accumulator out of
// tensor memory 16 columns at a time and store their rows between tiles.  Whether tensor memory's
// rate or that order bounds them is not known.)  One token: 14 us, 7.4 for the bytes at a copy's
// rate.
#include "layer.cuh"
#include "linear_rotate.cuh"
#include "tc.cuh"
#include "tensor_map.cuh"

namespace exl3 {

namespace {

using namespace tc;

__device__ unsigned int g_linear8_timeouts;

struct Args8 {
    const float *xs;
    int64_t xs_t, xs_b;
    const float *ws;
    int ws_o, ws_k;          // steps between the scales of neighbouring outputs and inputs
    int T;
    int n_out, blocks_k;     // outputs, blocks of 128 inputs
    int split;               // blocks of a cluster
    int tiles_t, tiles_f;    // tiles along tokens and outputs
    void *y;
    int dt;
    int64_t y_stride;
    bool behind;
};

// TN: columns of a tile (tokens with SWAP, else outputs); MN: W's rows run along its outputs
template <int TN, bool SWAP, bool MN> struct Form {
    static constexpr int kHalves = TN == 16 ? 1 : 2, kCols = TN / kHalves;     // columns of a result warp
    static constexpr int kOutWarps = 4 * kHalves, kThreads8 = (kOutWarps + 3) * 32;
    static constexpr int kCopy = kOutWarps, kIssue = kOutWarps + 1, kFactor = kOutWarps + 2;   // warps
    // results of a step in tensor memory: kAcc of them; what a block takes of it goes with
    // what it takes of shared memory (128 columns with more than a quarter, 512 with all but
    // 56 KB), so that blocks that fit an SM together never wait for each other's
    static constexpr int kAcc = SWAP ? 128 / TN : 512 / TN, kTmem = SWAP ? 128 : 512;
    static constexpr uint32_t kA = 16384, kB = TN * 128, kStage = kA + kB;
    static constexpr int kStages = SWAP ? 4 : TN == 128 ? 6 : 4;
    static constexpr uint32_t kSums = TN * 512;                                // split: the block's sums
    // factors of kFac steps, a product of scales for each token (SWAP) or token and 128 outputs;
    // a place of 32 tokens x 32 outputs for each result warp on their way out
    static constexpr int kFac = 8;
    static constexpr uint32_t kFacAt = kStages * kStage, kOutAt = kFacAt + kFac * TN * 4;
    static constexpr uint32_t kSmem = kOutAt + (SWAP ? 0u : kOutWarps * 2048u) + 1024;
    static_assert(kSums <= kStages * kStage, "sums in the place of the stages");
    static_assert(SWAP ? kSmem > 57 * 1024 && kSmem < 113 * 1024 : kSmem > 171 * 1024, "shared memory keeps tensor memory apart");
};

template <int COLS> __device__ __forceinline__ void tmem_alloc(uint32_t dst) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS> __device__ __forceinline__ void tmem_free(uint32_t addr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS));
}

// 16 columns of this warp's 32 lanes, asked for; they are there after the next tmem_wait
__device__ __forceinline__ void tmem_ask16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// e4m3 operands, binary32 accumulators; a_mn, b_mn: the operand's rows run along M or N
__device__ __forceinline__ uint32_t shape_e4m3(int m, int n, bool a_mn, bool b_mn) {
    return 1u << 4 | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
                 : "memory");
}

// a tile of a tensor map; the innermost coordinate is a multiple of 128 bytes
__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

// acc <- acc + f d for two neighbours
__device__ __forceinline__ void add_scaled(float &a0, float &a1, float f0, float f1, uint32_t d0, uint32_t d1) {
    asm("{\n\t.reg .b64 a, d, f;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 f, {%2, %3};\n\t"
        "mov.b64 d, {%4, %5};\n\t"
        "fma.rn.f32x2 a, d, f, a;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1) : "f"(f0), "f"(f1), "r"(d0), "r"(d1));
}

__device__ __forceinline__ uint32_t pack_dt(int dt, float a, float b) {
    return dt == EXL3_BF16 ? pack2<__nv_bfloat16>(a, b) : pack2<__half>(a, b);
}

template <int TN, bool SWAP, bool MN>
__global__ void __launch_bounds__(Form<TN, SWAP, MN>::kThreads8, SWAP ? 2 : 1)
    linear8_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ Args8 a) {
    using F = Form<TN, SWAP, MN>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[2 * F::kStages + 2 * F::kAcc + 2 * F::kFac + 1];
    __shared__ uint32_t tmem_at;
    __shared__ int gave_up;
    const uint32_t base = (saddr(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar0 = saddr(bars);
    auto full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8u * (F::kStages + s); };
    auto acc_full = [&](uint32_t d) { return bar0 + 8u * (2 * F::kStages + d); };
    auto acc_empty = [&](uint32_t d) { return bar0 + 8u * (2 * F::kStages + F::kAcc + d); };
    auto fac_full = [&](uint32_t d) { return bar0 + 8u * (2 * F::kStages + 2 * F::kAcc + d); };
    auto fac_empty = [&](uint32_t d) { return bar0 + 8u * (2 * F::kStages + 2 * F::kAcc + F::kFac + d); };
    const uint32_t drained = bar0 + 8u * (2 * F::kStages + 2 * F::kAcc + 2 * F::kFac);
    unsigned char *const sb = smem_raw + (base - saddr(smem_raw));
    float *const factors = reinterpret_cast<float *>(sb + F::kFacAt);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = a.split > 1 ? (int)(blockIdx.x % a.split) : 0;
    unsigned int *const count = &g_linear8_timeouts;

    if (tid == 0) {
        for (int s = 0; s < F::kStages; s++) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int d = 0; d < F::kAcc; d++) {
            bar_init(acc_full(d), 1);
            bar_init(acc_empty(d), F::kOutWarps);
        }
        for (int d = 0; d < F::kFac; d++) {
            bar_init(fac_full(d), 1);
            bar_init(fac_empty(d), F::kOutWarps);
        }
        bar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        gave_up = 0;
    }
    if (warp == F::kIssue)
        tmem_alloc<F::kTmem>(saddr(&tmem_at));
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_at;

    // tiles of this block, and its share of the inputs; a tile's number counts tokens first,
    // so that blocks running side by side share their weights
    const int tiles = a.tiles_t * a.tiles_f;
    const int it0 = (int)blockIdx.x / a.split, dit = a.split > 1 ? tiles : (int)gridDim.x;
    const int k_lo = a.blocks_k * rank / a.split, k_hi = a.blocks_k * (rank + 1) / a.split;
    const int steps = k_hi - k_lo;
    constexpr int kRowsT = SWAP ? TN : 128, kRowsF = SWAP ? 128 : TN;          // tokens and outputs of a tile
    auto t_of = [&](int it) { return it % a.tiles_t * kRowsT; };     // (2^24 tokens at most)
    auto f_of = [&](int it) { return it / a.tiles_t * kRowsF; };
    uint32_t issued = 0;                   // stages filled (of the thread that copies)

    if (warp == F::kCopy) {
        // ---- tiles of both operands, a stage for each 128 inputs ----
        if (elect()) {
            auto load_x = [&](uint32_t s, int t0, int k) {
                tile_load(base + s * F::kStage + (SWAP ? F::kA : 0u), &xmap, k * 128, t0, full(s));
            };
            auto load_w = [&](uint32_t s, int f0, int k) {
                const uint32_t to = base + s * F::kStage + (SWAP ? 0u : F::kA);
#pragma unroll
                for (int i = 0; i < kRowsF / 128; i++) {
                    if (MN)
                        tile_load(to + i * 16384u, &wmap, f0 + 128 * i, k * 128, full(s));
                    else
                        tile_load(to + i * 16384u, &wmap, k * 128, f0 + 128 * i, full(s));
                }
            };
            // the weights of the first stages need not wait for the launch before this one
            uint32_t ahead = 0;
            if (a.behind && it0 < tiles) {
                for (; ahead < F::kStages && (int)ahead < steps; ahead++) {
                    bar_expect(full(ahead), F::kStage);
                    load_w(ahead, f_of(it0), k_lo + (int)ahead);
                }
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            uint32_t s = 0, phase = 1;     // (the phase before the first is over)
            bool ok = true;
            for (int it = it0; ok && it < tiles; it += dit) {
                const int t0 = t_of(it);
                const int f0 = f_of(it);
                for (int k = k_lo; k < k_hi; k++) {
                    if (!bar_wait(empty(s), phase, &gave_up, count)) {
                        ok = false;
                        break;
                    }
                    if (issued >= ahead) {
                        bar_expect(full(s), F::kStage);
                        load_w(s, f0, k);
                    }
                    load_x(s, t0, k);
                    issued++;
                    if (++s == F::kStages)
                        s = 0, phase ^= 1;
                }
            }
            if (gave_up) {
                // nothing may be in flight when the block ends (a stage whose second copy was
                // never asked for does not end: the wait is bounded, as its first copy is done by then)
                const uint32_t most = issued > ahead ? issued : ahead;
                for (uint32_t back = 1; back <= F::kStages && back <= most; back++)
                    bar_drain(full((most - back) % F::kStages), ((most - back) / F::kStages) & 1);
            }
        }
    } else if (warp == F::kIssue) {
        // ---- matrix instructions ----
        if (elect()) {
            const bool a_mn = SWAP && MN, b_mn = !SWAP && MN;
            const uint32_t shape = shape_e4m3(128, TN, a_mn, b_mn);
            // 32 inputs on: 32 bytes of a row along K, or 32 rows
            constexpr uint32_t kHopA = (SWAP && MN ? 4096u : 32u) >> 4, kHopB = (!SWAP && MN ? 4096u : 32u) >> 4;
            uint32_t s = 0, s_phase = 0, d = 0, d_phase = 1;
            for (int it = it0; it < tiles && !gave_up; it += dit) {
                for (int k = 0; k < steps; k++) {
                    if (!bar_wait(acc_empty(d), d_phase, &gave_up, count) || !bar_wait(full(s), s_phase, &gave_up, count))
                        break;
                    fence_after();
                    const uint64_t da = operand(base + s * F::kStage, 16, 1024);
                    const uint64_t db = operand(base + s * F::kStage + F::kA, b_mn ? 16384 : 16, 1024);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        mma_e4m3(tmem + d * TN, da + i * kHopA, db + i * kHopB, shape, i > 0);
                    commit<false>(empty(s));
                    commit<false>(acc_full(d));
                    if (++s == F::kStages)
                        s = 0, s_phase ^= 1;
                    if (++d == F::kAcc)
                        d = 0, d_phase ^= 1;
                }
            }
            if (gave_up) {
                commit<false>(drained);
                bar_drain(drained, 0);
            }
        }
    } else if (warp == F::kFactor) {
        // ---- products of the scales: four steps on their way while four are written ----
        constexpr int kEach = SWAP ? (TN + 31) / 32 : 4, kBlocks = SWAP ? 1 : TN / 128, kTogether = 4;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        uint32_t s = 0, phase = 1;
        bool ok = true;
        for (int it = it0; ok && it < tiles; it += dit) {
            const int t0 = t_of(it) + lane, f0 = f_of(it);
            float x[kTogether][kEach], w[kTogether][kBlocks];
            auto ask = [&](int k0) {
#pragma unroll
                for (int j = 0; j < kTogether; j++) {
#pragma unroll
                    for (int i = 0; i < kEach; i++)
                        x[j][i] = k0 + j < steps && t0 + 32 * i < a.T && lane < TN
                                      ? __ldcg(a.xs + (int64_t)(t0 + 32 * i) * a.xs_t + (k_lo + k0 + j) * a.xs_b) : 0.0f;
#pragma unroll
                    for (int b = 0; b < kBlocks; b++)
                        w[j][b] = k0 + j < steps ? __ldg(a.ws + (int64_t)(min(f0 + 128 * b, a.n_out - 1) >> 7) * a.ws_o +
                                                         (int64_t)(k_lo + k0 + j) * a.ws_k) : 0.0f;
                }
            };
            ask(0);
            for (int k0 = 0; ok && k0 < steps; k0 += kTogether) {
                float f[kTogether][kBlocks][kEach];
#pragma unroll
                for (int j = 0; j < kTogether; j++)
#pragma unroll
                    for (int b = 0; b < kBlocks; b++)
#pragma unroll
                        for (int i = 0; i < kEach; i++)
                            f[j][b][i] = __fmul_rn(x[j][i], w[j][b]);
                ask(k0 + kTogether);
#pragma unroll
                for (int j = 0; j < kTogether; j++) {
                    if (!ok || k0 + j >= steps)
                        break;
                    ok = __all_sync(0xffffffffu, bar_wait(fac_empty(s), phase, &gave_up, count));
#pragma unroll
                    for (int b = 0; b < kBlocks; b++)
#pragma unroll
                        for (int i = 0; i < kEach; i++)
                            if (lane < TN)
                                factors[s * TN + b * 128 + 32 * i + lane] = f[j][b][i];
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(fac_full(s));
                    if (++s == F::kFac)
                        s = 0, phase ^= 1;
                }
            }
        }
    } else {
        // ---- results ----
        const int quarter = warp & 3, half = warp >> 2;
        const int row = quarter * 32 + lane;             // of the tile: an output (SWAP) or a token
        const float *const mine = factors + (SWAP ? half * F::kCols : half * F::kCols / 128 * 128 + row);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        uint32_t d = 0, d_phase = 0, s = 0, s_phase = 0;
        bool ok = true;
        for (int it = it0; ok && it < tiles; it += dit) {
            const int t0 = t_of(it);
            const int f0 = f_of(it);
            float acc[F::kCols];
#pragma unroll
            for (int c = 0; c < F::kCols; c++)
                acc[c] = 0.0f;
            for (int k = 0; k < steps; k++) {
                ok = __all_sync(0xffffffffu, bar_wait(fac_full(s), s_phase, &gave_up, count) && bar_wait(acc_full(d), d_phase, &gave_up, count));
                if (!ok)
                    break;
                fence_after();
                const uint32_t from = tmem + (uint32_t)(quarter * 32) * 65536u + d * TN + half * F::kCols;
                const float f = SWAP ? 0.0f : mine[s * TN];
                uint32_t r[2][16];
                tmem_ask16(from, r[0]);
#pragma unroll
                for (int c = 0; c < F::kCols; c += 16) {
                    uint32_t(&now)[16] = r[(c >> 4) & 1];
                    tmem_wait(now);
                    if (c + 16 < F::kCols)
                        tmem_ask16(from + c + 16, r[((c >> 4) + 1) & 1]);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        float4 g = make_float4(f, f, f, f);
                        if (SWAP)
                            g = *reinterpret_cast<const float4 *>(mine + s * TN + c + i);
                        add_scaled(acc[c + i], acc[c + i + 1], g.x, g.y, now[i], now[i + 1]);
                        add_scaled(acc[c + i + 2], acc[c + i + 3], g.z, g.w, now[i + 2], now[i + 3]);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(acc_empty(d));
                    bar_arrive(fac_empty(s));
                }
                if (++d == F::kAcc)
                    d = 0, d_phase ^= 1;
                if (++s == F::kFac)
                    s = 0, s_phase ^= 1;
            }
            if (!ok)
                break;
            if (a.split > 1) {
                // every step's operands have been used: their place takes the sums, by column
                float *const sums = reinterpret_cast<float *>(sb);
#pragma unroll
                for (int c = 0; c < F::kCols; c++)
                    sums[(half * F::kCols + c) * 128 + row] = acc[c];
            } else if (SWAP) {
                const int f = f0 + row;
#pragma unroll
                for (int c = 0; c < F::kCols; c++) {
                    const int t = t0 + half * F::kCols + c;
                    if (f < a.n_out && t < a.T)
                        reinterpret_cast<uint16_t *>(a.y)[(int64_t)t * a.y_stride + f] = (uint16_t)pack_dt(a.dt, acc[c], 0.0f);
                }
            } else {
                // 32 outputs of the warp's 32 tokens at a time, through shared memory: eight of a
                // token are 16 bytes, and a token's four such stand turned by its number
                uint4 *const place = reinterpret_cast<uint4 *>(sb + F::kOutAt) + warp * 128;
                const bool wide = (((uintptr_t)a.y | (uintptr_t)(a.y_stride * 2)) & 15u) == 0;
#pragma unroll
                for (int c = 0; c < F::kCols; c += 32) {
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const float *v = acc + c + 8 * u;
                        place[lane * 4 + (u ^ ((lane >> 1) & 3))] =
                            make_uint4(pack_dt(a.dt, v[0], v[1]), pack_dt(a.dt, v[2], v[3]), pack_dt(a.dt, v[4], v[5]), pack_dt(a.dt, v[6], v[7]));
                    }
                    __syncwarp();
                    const int f = f0 + half * F::kCols + c + (lane & 3) * 8;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int r = (lane >> 2) + 8 * j, t = t0 + quarter * 32 + r;
                        const uint4 q = place[r * 4 + ((lane & 3) ^ ((r >> 1) & 3))];
                        if (t < a.T && f < a.n_out) {    // (a multiple of 16)
                            uint16_t *y = reinterpret_cast<uint16_t *>(a.y) + (int64_t)t * a.y_stride + f;
                            if (wide) {
                                *reinterpret_cast<uint4 *>(y) = q;
                            } else {
                                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                                for (int i = 0; i < 8; i++)
                                    y[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }
    __syncwarp();

    if (a.split > 1) {
        // the blocks' sums, added in block order: groups of 8 columns, 32 rows a warp
        cluster_sync();
        const int t0 = t_of(it0);
        const int f0 = f_of(it0);
        const bool wide = (((uintptr_t)a.y | (uintptr_t)(a.y_stride * 2)) & 15u) == 0;
        constexpr int kWarps8 = F::kThreads8 / 32;
        if (SWAP) {
            // a column is a token: a lane takes four outputs of it
            for (int c = rank + warp * a.split; c < TN && t0 + c < a.T; c += kWarps8 * a.split) {
                float4 v = {};
                for (int b = 0; b < a.split; b++) {
                    float4 u;
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w)
                                 : "r"(at_block(base, b) + (uint32_t)(c * 128 + lane * 4) * 4u));
                    v.x = __fadd_rn(v.x, u.x), v.y = __fadd_rn(v.y, u.y), v.z = __fadd_rn(v.z, u.z), v.w = __fadd_rn(v.w, u.w);
                }
                const int f = f0 + lane * 4;
                if (f < a.n_out) {
                    uint16_t *y = reinterpret_cast<uint16_t *>(a.y) + (int64_t)(t0 + c) * a.y_stride + f;
                    const uint32_t q[2] = {pack_dt(a.dt, v.x, v.y), pack_dt(a.dt, v.z, v.w)};
                    if (wide) {
                        *reinterpret_cast<uint2 *>(y) = make_uint2(q[0], q[1]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            y[i] = (uint16_t)(q[i >> 1] >> (16 * (i & 1)));
                    }
                }
            }
        } else {
            // a column is an output: a lane takes eight of its token
            for (int u = rank + warp * a.split; u < TN / 8 * 4; u += kWarps8 * a.split) {
                const int c = u >> 2 << 3, row = (u & 3) * 32 + lane;
                const int t = t0 + row;
                const int f = f0 + c;
                if (t0 + (u & 3) * 32 >= a.T || f >= a.n_out)
                    continue;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[i] = 0.0f;
                for (int b = 0; b < a.split; b++) {
                    const uint32_t from = at_block(base, b) + (uint32_t)(c * 128 + row) * 4u;
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        float w;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(from + i * 512u));
                        v[i] = __fadd_rn(v[i], w);
                    }
                }
                if (t < a.T) {
                    uint16_t *y = reinterpret_cast<uint16_t *>(a.y) + (int64_t)t * a.y_stride + f;
                    uint32_t q[4];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        q[i] = pack_dt(a.dt, v[2 * i], v[2 * i + 1]);
                    if (wide) {
                        *reinterpret_cast<uint4 *>(y) = make_uint4(q[0], q[1], q[2], q[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            y[i] = (uint16_t)(q[i >> 1] >> (16 * (i & 1)));
                    }
                }
            }
        }
        cluster_sync();                    // no block ends while another may still read its sums
    }
    fence_before();
    __syncthreads();
    if (warp == F::kIssue) {
        fence_after();
        tmem_free<F::kTmem>(tmem);
    }
}

// row-major [rows, cols] bytes; boxes of 128 columns, one swizzled row of an operand each
bool encode_bytes(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t each[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, each,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TN, bool SWAP, bool MN> exl3_status launch_form8(const Linear8Launch &p, Args8 &a, cudaStream_t s) {
    using F = Form<TN, SWAP, MN>;
    constexpr int kRowsT = SWAP ? TN : 128, kRowsF = SWAP ? 128 : TN;
    const int64_t sms = device_sm_count();
    a.tiles_t = (a.T + kRowsT - 1) / kRowsT;
    a.tiles_f = (a.n_out + kRowsF - 1) / kRowsF;
    const int64_t tiles = (int64_t)a.tiles_t * a.tiles_f, slots = SWAP ? 2 * sms : sms;
    // blocks that would idle share the inputs of the tiles, two steps each at least (one or four at
    // least are as fast: 512 -> 512 7.2, 6.7 and 6.7 us).  One token, replayed graphs, us, not split
    // and 2, 4, 8 blocks to a tile, the rule's choice in brackets: 4096 -> 12288 17.8 (16.3) 15.8 18.5;
    // 4096 -> 4096 13.3 10.8 8.8 (9.7); 12288 -> 4096 34.6 22.6 16.8 (15.5); 4096 -> 1024 12.7 10.3 8.2 (8.2)
    a.split = 1;
    while (a.split < 8 && tiles * a.split * 2 <= slots && a.blocks_k >= a.split * 4)
        a.split *= 2;
    CUtensorMap xmap, wmap;
    if (!encode_bytes(&xmap, p.x, p.T, p.transposed ? p.cols : p.rows, p.x_stride, kRowsT) ||
        !encode_bytes(&wmap, p.w, p.rows, p.cols, p.cols, 128))
        return set_error(EXL3_ERR_CUDA, "no tensor map for the operands");
    cudaError_t e = allow_smem((const void *)linear8_kernel<TN, SWAP, MN>, F::kSmem);
    if (e != cudaSuccess)
        return cuda_check(e, "cudaFuncSetAttribute(8-bit product)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.split > 1 ? tiles * a.split : tiles < slots ? tiles : slots));
    cfg.blockDim = dim3(F::kThreads8);
    cfg.dynamicSmemBytes = F::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.behind ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, linear8_kernel<TN, SWAP, MN>, xmap, wmap, a);
    if (e != cudaSuccess)
        return cuda_check(e, "8-bit product launch");
    note_launch();
    return cuda_check(cudaGetLastError(), "8-bit product launch");
}

// Outputs are the instruction's rows up to 64 tokens: replayed graphs, us, 4096 x 4096, outputs / tokens as
// rows: 17 tokens 10.3 / 12.4, 32 10.3 / 11.3, 64 12.3 / 12.2, 65 13.4 / 12.4.  256 outputs a tile where tiles
// fill the SMs, else 128: 4096 tokens x 4096 x 12288 181 and 202, 2048 x 4096 x 4096 39 and 45.
template <bool MN> exl3_status launch_mn(const Linear8Launch &p, Args8 &a, cudaStream_t s) {
    if (a.T <= 16)
        return launch_form8<16, true, MN>(p, a, s);
    if (a.T <= 32)
        return launch_form8<32, true, MN>(p, a, s);
    if (a.T <= 64)
        return launch_form8<64, true, MN>(p, a, s);
    const int64_t tiles = (int64_t)((a.T + 127) / 128) * ((a.n_out + 255) / 256);
    return tiles >= device_sm_count() ? launch_form8<256, false, MN>(p, a, s) : launch_form8<128, false, MN>(p, a, s);
}

}  // namespace

exl3_status launch_linear8(const Linear8Launch &p, cudaStream_t s) {
    Args8 a = {};
    const int64_t n_in = p.transposed ? p.cols : p.rows;
    const int blocks_c = (int)((p.cols + 127) / 128);
    a.xs = p.xs;
    a.xs_t = p.xs_t;
    a.xs_b = p.xs_b;
    a.ws = p.ws;
    a.ws_o = p.transposed ? blocks_c : 1;
    a.ws_k = p.transposed ? 1 : blocks_c;
    a.T = (int)p.T;
    a.n_out = (int)(p.transposed ? p.rows : p.cols);
    a.blocks_k = (int)((n_in + 127) / 128);
    a.y = p.y;
    a.dt = p.dt;
    a.y_stride = p.y_stride;
    a.behind = p.behind;
    return p.transposed ? launch_mn<false>(p, a, s) : launch_mn<true>(p, a, s);
}

exl3_status linear8_take_wait_timeouts(unsigned int *n) {
    *n = 0;
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_linear8_timeouts, sizeof v);
    if (e == cudaSuccess && v != 0)
        e = cudaMemcpyToSymbol(g_linear8_timeouts, &zero, sizeof zero);
    if (e != cudaSuccess)
        return cuda_check(e, "wait timeout count");
    *n = v;
    return EXL3_OK;
}

}  // namespace exl3
