// linear_product.cu -- y = z V H . right . 2^-7 s (see linear.cuh) with V decoded
// from the codes on the way into the tensor cores.
//
// The product runs transposed: a block owns 128 outputs (the lanes of its
// accumulators) and the tokens are the columns, so that a weight is decoded
// once for many tokens and a single token still fills every lane.  Warps have
// roles:
//   0-15   decode, eight warps to a 128 x 64 step and taking turns: 32 weights a
//          thread to a swizzled operand stage.  The weights of a tile row run
//          along the outputs (x W^) or along the sum (x W^^T): the first is
//          stored as an operand whose rows run along M, the second along K, and
//          only the descriptor differs;
//   16-23  results, two groups that take turns at chunks of 32 tokens: accumulator ->
//          shared memory (one token per row) -> H over the 128 outputs in two passes ->
//          scales, adapters, one rounding (3000 cycles a chunk; with one group of four
//          the last tile's results stood alone twice as long);
//   24     bulk copies of the rotated activations, one contiguous block a step;
//   25     issues the matrix instructions (binary16 in, binary32 out).
//
// Two forms.  Alone, a block multiplies by up to 256 tokens and two
// accumulators let the results of one tile overlap the sums of the next.  In
// pairs (PAIR, a cluster of two), one instruction multiplies the 256 outputs of
// both blocks by up to 256 tokens of which each block holds half, and a tile
// has up to 512 tokens in two accumulators: each weight is decoded for twice
// the tokens, and each copy of activations feeds twice the outputs.
//
// Bound: of a step's cycles the decode takes 384 of each quarter's arithmetic pipes,
// the matrix instructions 512 for 256 tokens (1024 for a pair's 512), and shared memory
// about 900 in a pair (writing and reading both operands); measured are 1000 a step, up
// to 480 tokens in a pair, because the roles share the issue slots and the shared
// memory.  4096 x 4096 x 4096, K = 2, in pairs: 119 us with the rotation before it, and
// the kernel alone 122 to 125 where it adds adapters' terms (64 MB more to read, which the
// ends of its two rounds wait for); 1001 tokens x 4096 x 4096, K = 4, with terms: 48 us.
//
// With few tiles (decode), the sum is split over the `split` blocks of a
// cluster; each leaves its partial sums in its shared memory and block r adds
// up, in block order, and finishes tokens r, r + split, ...
//
// Every wait is bounded (tc.cuh); after one gives up the block stops issuing,
// waits for what it has in flight, and its results are void (counted in
// exl3_wait_timeouts).
#include "linear_decode.cuh"
#include "tc.cuh"

namespace exl3 {

namespace {

using namespace tc;

constexpr int kGroups = 2, kDecWarps = 8 * kGroups, kOutWarps = 8;
constexpr int kWarpB = kDecWarps + kOutWarps, kWarpMma = kWarpB + 1;
constexpr int kThreadsP = (kWarpB + 2) * 32;
constexpr int kN = 256;                    // columns of an accumulator
constexpr int kStep = 64;                  // inputs of a step
constexpr int kAStages = 3, kBStages = 16; // operand stages (of B at most; a fourth of A changed no time)
constexpr uint32_t kABytes = 128 * kStep * 2, kBArea = 96 * 1024, kCArea = 16 * 1024;
constexpr uint32_t kBOff = kAStages * kABytes;              // B stages behind the A stages,
constexpr uint32_t kCOff = kBOff + kBArea;                  // then a ring of codes for each decode warp,
constexpr uint32_t kOutOff = kCOff + kCArea;                // then 32 tokens x 128 outputs, fp32, for four result warps each,
constexpr uint32_t kAddOff = kOutOff + 2 * 32 * 128 * 4;    // then 128 bytes for each of their threads,
constexpr uint32_t kPlanOff = kAddOff;                      // or the experts' tiles (which have no adapters)
constexpr uint32_t kSmem = kAddOff + 256 * 128 + 1024;      // + alignment slack
static_assert(sizeof(Plan) <= 256 * 128, "the plan fits where the adapters' terms would be");

__device__ unsigned int g_product_timeouts;

// 16-bit window `sh` bits before the end of r.  Byte-aligned picks share one
// funnel shift for each bit offset.
template <int NR> __device__ __forceinline__ uint32_t window(const uint32_t (&r)[NR], int sh) {
    const int a = NR - 1 - (sh >> 5), b = sh & 31;
    const uint32_t hi = a > 0 ? r[a > 0 ? a - 1 : 0] : 0u;
    if (b < 24) {
        const uint32_t f = (b & 7) ? __funnelshift_r(r[a], hi, b & 7) : r[a];
        return __byte_perm(f, 0u, b < 8 ? 0x4410 : b < 16 ? 0x4421 : 0x4432);
    }
    return __funnelshift_r(r[a], hi, b) & 0xFFFFu;
}

// A row of 16 weights, to the 32 bytes of an operand row at `to` (the second 16 at
// to ^ 16).  The row's windows need the 15 + 16 K bits up to its last one: NR words that
// end with it, from NL words of the tile, the last at `last`, the first at `first` (the
// stream is a ring; only the first can be around it).  `half`: 16 where the row ends in
// the middle of a word (odd K).
template <int K> struct Row {
    static constexpr int NR = (15 + 16 * K + 31) / 32, NL = (K & 1) ? NR + 1 : NR;
    uint32_t last, first, half, to;
    // row R of a tile at offset `tile` of the codes, column 16 tc of an operand panel at `panel`
    __device__ __forceinline__ Row(uint32_t tile, uint32_t panel, int R, int tc) {
        const int end = 16 * K * (R + 1), w = (end - 1) >> 5, f = w - (NL - 1);
        last = tile + 4u * w;
        first = tile + 4u * (f < 0 ? f + 8 * K : f);
        half = end & 16;
        to = panel + R * 128 + (((2 * tc) ^ (R & 7)) << 4);
    }
};
template <int K> __device__ __forceinline__ void decode_row(const Row<K> &row, uint32_t codes, uint32_t stage) {
    constexpr int NR = Row<K>::NR, NL = Row<K>::NL;
    uint32_t l[NL], r[NR];
#pragma unroll
    for (int j = 0; j < NL; j++)
        asm volatile("ld.shared.b32 %0, [%1];"
                     : "=r"(l[j]) : "r"(j == 0 ? codes + row.first : codes + row.last - 4u * (NL - 1 - j)));
#pragma unroll
    for (int j = 0; j < NR; j++)
        r[j] = (K & 1) ? __funnelshift_r(l[j + NL - NR], l[j + NL - NR - (K & 1)], row.half) : l[j];
    const uint32_t to = stage + row.to;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        uint32_t v[4];
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const int c = 8 * h + 2 * p;
            v[p] = levels2(window<NR>(r, (15 - c) * K), window<NR>(r, (14 - c) * K));
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to ^ (h << 4)), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3])
                     : "memory");
    }
}

struct Tile : OutTile<int> {
    int n;            // columns, a multiple of 16 (PAIR: 32)
};

struct Args {
    ProductLaunch p;
    int n_in, n_out;
    int tile_n;          // tokens of a tile (a multiple of 16 up to 256, PAIR: of 32 up to 512)
    int b_steps;         // steps of a B stage: the fewer the tokens, the more
    int b_stages;        // B stages of b_steps steps of tile_n tokens (PAIR: of half of them)
    int split;           // blocks of a cluster, each with its share of the steps
};

// The second block of the last pair may have no outputs (f0 == n_out).
template <bool PAIR> __device__ __forceinline__ Tile make_tile(const Args &a, const Plan *plan, int64_t it, int rank) {
    Tile t;
    static_cast<OutTile<int> &>(t) =
        out_tile<int>(a.p.offsets ? plan : nullptr, a.p.E, (int)a.p.T, a.tile_n, PAIR ? (a.n_out / 128 + 1) / 2 : a.n_out / 128,
                 PAIR ? 256 : 128, it);
    if (PAIR)
        t.f0 += rank * 128;
    t.n = PAIR ? (t.hi - t.t0 + 31) / 32 * 32 : (t.hi - t.t0 + 15) / 16 * 16;
    return t;
}

// right . 2^-7 s of output f < 128 of the tile
__device__ __forceinline__ float right_of(const Args &a, const Tile &tl, int f) {
    const int f0 = min(tl.f0, a.n_out - 128);
    return __fmul_rn(__ldg(a.p.right + (size_t)tl.e * a.n_out + f0 + f), __fmul_rn(__ldg(a.p.scale + tl.e), 0x1p-7f));
}

template <int K, bool PAIR, typename TY>
__global__ void __launch_bounds__(kThreadsP, 1) product_kernel(const __grid_constant__ Args a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[2 * kAStages + 2 * kBStages + 5];
    __shared__ __align__(16) float rights[2][128];
    __shared__ uint32_t tmem_at;
    __shared__ int gave_up;
    const uint32_t base = (saddr(smem_raw) + 1023u) & ~1023u;
    unsigned char *const sb = smem_raw + (base - saddr(smem_raw));
    Plan &plan = *reinterpret_cast<Plan *>(sb + kPlanOff);
    const uint32_t bar_a = saddr(bars), bar_b = bar_a + 16u * kAStages;
    const uint32_t bar_d = bar_b + 16u * kBStages;
    auto full_a = [&](uint32_t s) { return bar_a + 8u * s; };
    auto empty_a = [&](uint32_t s) { return bar_a + 8u * (kAStages + s); };
    auto full_b = [&](uint32_t s) { return bar_b + 8u * s; };
    auto empty_b = [&](uint32_t s) { return bar_b + 8u * (kBStages + s); };
    auto acc_full = [&](uint32_t i) { return bar_d + 8u * i; };
    auto acc_empty = [&](uint32_t i) { return bar_d + 8u * (2 + i); };
    const uint32_t drained = bar_d + 32u;
    // (through a shuffle the compiler knows the warp's number, and what follows from it, as uniform)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = PAIR ? (int)(blockIdx.x & 1) : a.split > 1 ? (int)(blockIdx.x % a.split) : 0;

    if (tid == 0) {
        for (int s = 0; s < kAStages; s++) {
            bar_init(full_a(s), PAIR ? 16 : 8);
            bar_init(empty_a(s), 1);
        }
        for (int s = 0; s < kBStages; s++) {
            bar_init(full_b(s), 1);
            bar_init(empty_b(s), 1);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(acc_full(i), 1);
            bar_init(acc_empty(i), PAIR ? 2 * kOutWarps : kOutWarps);
        }
        bar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        gave_up = 0;
    }
    if (warp == kDecWarps)
        tmem_alloc_all<PAIR>(saddr(&tmem_at));
    if (a.p.offsets)
        make_plan(plan, a.p.offsets, a.p.E, a.p.T, a.tile_n, tid, kThreadsP);
    fence_before();
    __syncthreads();
    if (PAIR)
        cluster_sync();                    // the other block's barriers are ready
    fence_after();
    const uint32_t tmem = tmem_at;
    const int64_t n_tok = a.p.offsets ? plan.first[a.p.E] : (a.p.T + a.tile_n - 1) / a.tile_n;
    const int64_t n_tiles = n_tok * (PAIR ? (a.n_out / 128 + 1) / 2 : a.n_out / 128);
    const int blocks = PAIR ? 2 : a.split;                                             // of a cluster
    const int64_t it0 = blockIdx.x / blocks, dit = !PAIR && a.split > 1 ? n_tiles : gridDim.x / blocks;
    const int steps = a.n_in / kStep;
    const int k_lo = PAIR ? 0 : (int)((int64_t)steps * rank / a.split);
    const int k_hi = PAIR ? steps : (int)((int64_t)steps * (rank + 1) / a.split);
    const int64_t NP = act_rows(a.p.T);
    const uint32_t nb = (uint32_t)a.b_stages, b_step = (uint32_t)a.tile_n * (PAIR ? 64u : 128u);   // bytes of a step
    const uint32_t b_bytes = b_step * (uint32_t)a.b_steps;
    unsigned int *const count = &g_product_timeouts;
    const uint32_t n_mine = it0 < n_tiles ? (uint32_t)((n_tiles - 1 - it0) / dit + 1) : 0u;
    uint32_t issued = 0;                   // B stages copied (of the thread that copies)

    if (warp < kDecWarps) {
        // ---- decode: groups of eight warps take turns at the steps ----
        const int q = lane >> 2, tc = lane & 3, dw = warp & 7, group = warp >> 3, odd = q & 1;
        const uint32_t panel = a.p.transposed ? (uint32_t)dw * 16u * 128u
                                              : (uint32_t)(dw & 1) * 8192u + (uint32_t)(dw >> 1) * 16u * 128u;
        const uint32_t n = (uint32_t)(k_hi - k_lo), total = n_mine * n;
        // This warp's codes of a step are those of four neighbouring tiles, 128 K
        // bytes in a row.  They are copied kRing of its steps ahead, across tiles.
        constexpr uint32_t kSlot = 128 * K, kRing = kCArea / (kDecWarps * kSlot);
        static_assert(kRing * kSlot * kDecWarps <= kCArea, "code rings");
        const uint32_t ring = base + kCOff + (uint32_t)warp * (kRing * kSlot);
        const int64_t tiles_c = a.p.cols / 16;
        const int tr = a.p.transposed ? dw : dw >> 1, tcol = a.p.transposed ? 0 : (dw & 1) * 4;
        const int64_t hop = (a.p.transposed ? 4 : 4 * tiles_c) * (32 * K);       // bytes from step to step
        uint32_t k_load = group, left = total > (uint32_t)group ? (total - group + kGroups - 1) / kGroups : 0u, slot_load = 0;
        int64_t it_load = it0;
        const char *p_load = nullptr;      // codes of step k_load
        auto next_codes = [&]() {
            if (left) {
                left--;
                if (!p_load || k_load >= n) {
                    // another tile
                    if (p_load)
                        do
                            k_load -= n, it_load += dit;
                        while (k_load >= n);
                    else
                        for (; k_load >= n; k_load -= n)
                            it_load += dit;
                    const Tile tl = make_tile<PAIR>(a, &plan, it_load, rank);
                    const int f0 = PAIR ? min(tl.f0, a.n_out - 128) : tl.f0;
                    const int64_t r0 = a.p.transposed ? f0 / 16 + tr : (int64_t)k_lo * 4 + tr;
                    const int64_t c0 = a.p.transposed ? (int64_t)k_lo * 4 + tcol : f0 / 16 + tcol;
                    p_load = reinterpret_cast<const char *>(a.p.codes) +
                             ((int64_t)tl.e * (a.p.rows / 16) * tiles_c + r0 * tiles_c + c0) * (32 * K) + lane * 16 +
                             k_load * hop;
                }
                if (lane < 8 * K)
                    copy16(ring + slot_load * kSlot + lane * 16, p_load);
                p_load += kGroups * hop;
                k_load += kGroups;
            }
            copy_group();
            slot_load = slot_load + 1 == kRing ? 0 : slot_load + 1;
        };
#pragma unroll 1
        for (uint32_t i = 0; i < kRing; i++)
            next_codes();
        // This lane's rows 2q and 2q + 1 of tile tc.  Lanes of odd q take their second row
        // first: the eight lanes of a store phase then cover all banks.
        const Row<K> row0(tc * (32u * K), panel, 2 * q + odd, tc), row1(tc * (32u * K), panel, 2 * q + 1 - odd, tc);
        uint32_t codes = ring, stage = base + (uint32_t)(group % kAStages) * kABytes, s_b = group % nb, round_b = group / nb;
        uint32_t bar = full_a(group % kAStages), round = 0;       // (the stage's full barrier; the empty one lies kAStages behind)
#pragma unroll 1
        for (uint32_t i = total > (uint32_t)group ? (total - group + kGroups - 1) / kGroups : 0u; i; i--) {
            if (!__all_sync(0xffffffffu, round == 0 || bar_wait(bar + 8u * kAStages, (round - 1) & 1, &gave_up, count)))
                break;                     // the warp goes on as a whole or not at all
            copy_wait<kRing - 1>();
            __syncwarp();
            decode_row<K>(row0, codes, stage);
            decode_row<K>(row1, codes, stage);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (PAIR && rank == 1 && dw == 0) {
                // block 0 issues for both: this block's arrival also says that its activations have landed
                if (!__all_sync(0xffffffffu, bar_wait(full_b(s_b), round_b & 1, &gave_up, count)))
                    break;
                for (int j = 0; j < kGroups; j++)
                    if (++s_b == nb)
                        s_b = 0, round_b++;
            }
            if (lane == 0) {
                if (PAIR && rank == 1)
                    bar_arrive_at(at_block(bar, 0));
                else
                    bar_arrive(bar);
            }
            next_codes();
            codes += kSlot;
            if (codes == ring + kRing * kSlot)
                codes = ring;
            stage += kGroups * kABytes;
            bar += kGroups * 8u;
            if (stage >= base + kAStages * kABytes)
                stage -= kAStages * kABytes, bar -= kAStages * 8u, round++;
        }
    } else if (warp < kDecWarps + kOutWarps) {
        // ---- results ----
        // two groups of four warps take turns at the chunks of 32 tokens
        const int ow = warp & 3, og = (warp - kDecWarps) >> 2;
        float *const right = rights[og];
        const bool keep = !PAIR && a.split > 1;             // partial sums stay in shared memory
        float *const buf = reinterpret_cast<float *>(sb + (keep ? 0u : kOutOff + og * (32u * 128u * 4u)));
        const int f4 = 8 * ow + (lane >> 2), col = 4 * out_at(f4) + (lane & 3);
        const int col0 = 4 * swz(f4, 0) + (lane & 3), col1 = 4 * swz(f4, 1) + (lane & 3);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the adapters' gradients)
        uint32_t acc = 0;
        bool ok = true;
        const int u = lane & 7;
        for (int64_t it = it0; ok && it < n_tiles; it += dit) {
            const Tile tl = make_tile<PAIR>(a, &plan, it, rank);
            const bool live = !PAIR || tl.f0 < a.n_out;
            // read after the barriers of the first chunk; the last chunk's protect the previous tile's
            right[ow * 32 + lane] = right_of(a, tl, ow * 32 + lane);
            // A thread finishes two tokens of every 32, eight threads to a token.  What it
            // needs of them from memory is asked for a chunk before: the row's scale, and of a
            // token with an adapter its part of the result (to its own place in shared memory).
            float rs[2];
            bool more[2];
            const uint32_t mine = base + kAddOff + (uint32_t)og * 16384u + (uint32_t)(ow * 32 + lane) * 16u;
            auto fetch = [&](int g, int t) {
                const bool in = !keep && live && t >= tl.lo && t < tl.hi;
                rs[g] = in ? a.p.rscale[t] : 0.0f;
                more[g] = a.p.term && in && has_term(a.p, t);
                if (a.p.term && in) {
                    const float4 *from = term_at(a.p, a.n_out, tl.f0, t, u);
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        copy16(mine + (4 * g + q) * 2048u, from + (q & 1) + 16 * (q >> 1));
                }
                copy_group();
            };
            const int t_mine = tl.t0 + ow * 4 + (lane >> 3);
            fetch(0, t_mine + 32 * og);
            fetch(1, t_mine + 32 * og + 16);
            for (int n0 = 0; ok && n0 < tl.n; n0 += kN, acc++) {
                const int d = acc & 1;
                ok = bar_wait(acc_full(d), (acc >> 1) & 1, &gave_up, count);
                // the group goes on as a whole or not at all: another wait of the block may have
                // given up while this phase ended, and a warp that left would be missing below
                ok = bar_all(1 + og, 128, __all_sync(0xffffffffu, ok));
                if (!ok)
                    break;
                fence_after();
                const int n1 = min(tl.n - n0, kN);
                for (int c0 = 32 * og; c0 < n1; c0 += 64) {
#pragma unroll
                    for (int g = 0; g < 2; g++) {
                        float v[16];
                        tmem_load16(tmem + (uint32_t)(ow * 32) * 65536u + d * kN + c0 + 16 * g, v);
                        if (keep) {
#pragma unroll
                            for (int i = 0; i < 16; i++)
                                buf[(c0 + 16 * g + i) * 128 + col] = v[i];
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i++)
                                buf[(16 * g + i) * 128 + (i & 1 ? col1 : col0)] = v[i];
                        }
                    }
                    if (keep)
                        continue;
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + og) : "memory");
                    rotate_first(buf, ow * 32 + lane);
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + og) : "memory");
#pragma unroll
                    for (int g = 0; g < 2; g++) {
                        const int t = t_mine + n0 + c0 + 16 * g;
                        float x[16];
                        rotate_second(buf, g * 16 + ow * 4 + (lane >> 3), u, rs[g], right, x);
                        const bool in = live && t >= tl.lo && t < tl.hi;
                        copy_wait<1>();
                        if (more[g]) {     // (the thread's own copies: no barrier)
#pragma unroll
                            for (int q = 0; q < 4; q++) {
                                const float4 f = *reinterpret_cast<const float4 *>(sb + (mine - base) + (4 * g + q) * 2048);
                                x[4 * q] = __fadd_rn(x[4 * q], f.x), x[4 * q + 1] = __fadd_rn(x[4 * q + 1], f.y);
                                x[4 * q + 2] = __fadd_rn(x[4 * q + 2], f.z), x[4 * q + 3] = __fadd_rn(x[4 * q + 3], f.w);
                            }
                        } else if (a.p.B && in) {
                            add_adapter<TY>(a.p, a.n_out, tl.f0, t, x, u, 0, 1);
                        }
                        fetch(g, t + 64);
                        if (in)
                            store_out<TY>(a.p, tl.f0, t, x, u);
                    }
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + og) : "memory");
                }
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && rank == 1)
                        bar_arrive_at(at_block(acc_empty(d), 0));
                    else
                        bar_arrive(acc_empty(d));
                }
            }
        }
    } else if (warp == kWarpB) {
        // ---- activations ----
        asm volatile("griddepcontrol.wait;" ::: "memory");
        bool ok = true;
        uint32_t s = 0, phase = 1;         // (the phase before the first is over)
        for (int64_t it = it0; ok && it < n_tiles; it += dit) {
            const Tile tl = make_tile<PAIR>(a, &plan, it, rank);
            const unsigned char *src = a.p.image + ((int64_t)k_lo * NP + tl.t0) * 128;
            const int64_t hop = NP * 128;
            // PAIR: this block's half of the columns of each accumulator
            const uint32_t n1 = PAIR ? (uint32_t)min(tl.n, kN) * 64u : (uint32_t)tl.n * 128u;
            const uint32_t n2 = PAIR && tl.n > kN ? (uint32_t)(tl.n - kN) * 64u : 0u;
            const unsigned char *src1 = src + (PAIR ? (uint32_t)rank * n1 : 0u);
            const unsigned char *src2 = src + kN * 128 + (uint32_t)rank * n2;
            for (int k = k_lo; k < k_hi; k += a.b_steps) {
                if (!__all_sync(0xffffffffu, bar_wait(empty_b(s), phase, &gave_up, count))) {
                    ok = false;
                    break;
                }
                const int steps_here = min(a.b_steps, k_hi - k);
                if (elect()) {
                    uint32_t dst = base + kBOff + s * b_bytes;
                    bar_expect(full_b(s), (uint32_t)steps_here * (n1 + n2));
                    for (int j = 0; j < steps_here; j++, dst += b_step) {
                        bulk_load(dst, src1 + j * hop, n1, full_b(s));
                        if (PAIR && n2)
                            bulk_load(dst + kN * 64, src2 + j * hop, n2, full_b(s));
                    }
                }
                __syncwarp();
                src1 += steps_here * hop;
                src2 += steps_here * hop;
                issued++;
                if (++s == nb)
                    s = 0, phase ^= 1;
            }
        }
    } else if (!PAIR || rank == 0) {
        // ---- matrix instructions: one thread, as little around them as there can be ----
        if (elect()) {
            uint32_t acc = 0, s = 0, s_phase = 0, sa = 0, sa_phase = 0;
            // 16 inputs on: 32 bytes of a row along K, two groups of 8 rows along M
            const uint64_t a0 = a.p.transposed ? operand(base, 16, 1024) : operand(base, 8192, 1024);
            const uint64_t b0 = operand(base + kBOff, 16, 1024);
            const uint32_t hop_a = a.p.transposed ? 32 >> 4 : 2048 >> 4;
            const int b_steps = a.b_steps;
            uint64_t da = a0, db0 = b0;
            for (int64_t it = it0; it < n_tiles; it += dit) {
                const Tile tl = make_tile<PAIR>(a, &plan, it, rank);
                const bool two = PAIR && tl.n > kN;
                if (acc >= 2 && !bar_wait(acc_empty(acc & 1), ((acc >> 1) - 1) & 1, &gave_up, count))
                    break;
                if (two && acc + 1 >= 2 && !bar_wait(acc_empty((acc + 1) & 1), (((acc + 1) >> 1) - 1) & 1, &gave_up, count))
                    break;
                const uint32_t shape = shape_f16(PAIR ? 256 : 128, two ? kN : tl.n, !a.p.transposed);
                const uint32_t shape2 = shape_f16(256, tl.n - kN, !a.p.transposed);
                const uint32_t d = tmem + (acc & 1) * kN, d2 = tmem + ((acc + 1) & 1) * kN;
                int left = k_hi - k_lo;
                bool add = false;
                while (left > 0) {
                    if (!bar_wait(full_b(s), s_phase, &gave_up, count))
                        break;
                    int j = left < b_steps ? left : b_steps;
                    left -= j;
                    uint64_t db = db0;
                    for (; j; j--, db += b_step >> 4) {
                        if (!bar_wait(full_a(sa), sa_phase, &gave_up, count)) {
                            left = -1;
                            break;
                        }
                        fence_after();
#pragma unroll
                        for (int i = 0; i < kStep / 16; i++)
                            mma_f16<PAIR>(d, da + i * hop_a, db + i * 2, shape, add || i > 0);
                        if (two) {
#pragma unroll
                            for (int i = 0; i < kStep / 16; i++)
                                mma_f16<PAIR>(d2, da + i * hop_a, db + (kN * 64 >> 4) + i * 2, shape2, add || i > 0);
                        }
                        add = true;
                        commit<PAIR>(empty_a(sa));
                        da += kABytes >> 4;
                        if (++sa == kAStages)
                            sa = 0, sa_phase ^= 1, da = a0;
                    }
                    if (left < 0)
                        break;
                    commit<PAIR>(empty_b(s));
                    db0 += b_bytes >> 4;
                    if (++s == nb)
                        s = 0, s_phase ^= 1, db0 = b0;
                }
                if (gave_up)
                    break;
                commit<PAIR>(acc_full(acc & 1));
                if (two)
                    commit<PAIR>(acc_full((acc + 1) & 1));
                acc += two ? 2 : 1;
            }
        }
    }
    __syncwarp();

    if (!PAIR && a.split > 1) {
        // partial sums of the cluster, added in block order
        cluster_sync();
        if (it0 < n_tiles && warp < kDecWarps + kOutWarps) {
            const Tile tl = make_tile<PAIR>(a, &plan, it0, rank);
            // a warp takes four tokens at a time, with adapters one (its four groups of eight
            // lanes a quarter of the adapter's rows each)
            const bool shared = a.p.B != nullptr;
            const int each = shared ? 1 : 4, sub = shared ? 0 : lane >> 3, u = lane & 7;
            const int mine = (tl.n + a.split - 1 - rank) / a.split;          // tokens rank, rank + split, ...
            for (int i = warp * each; i < mine; i += (kDecWarps + kOutWarps) * each) {
                const int row = rank + (i + sub) * a.split;
                const bool in = row < tl.n;
                const int t = in ? tl.t0 + row : tl.hi;
                const float rs = t < tl.hi ? a.p.rscale[t] : 0.0f;
                float v[16], x[16];
#pragma unroll
                for (int j = 0; j < 16; j++)
                    v[j] = x[j] = 0.0f;
                if (shared && t >= tl.lo && t < tl.hi) {
                    add_adapter<TY>(a.p, a.n_out, tl.f0, t, v, u, lane >> 3, 4);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        v[j] = __fadd_rn(v[j], __shfl_xor_sync(0xffffffffu, v[j], 8));
                        v[j] = __fadd_rn(v[j], __shfl_xor_sync(0xffffffffu, v[j], 16));
                    }
                }
                if (in)
#pragma unroll 2
                    for (int b = 0; b < a.split; b++)
                        add_sums(x, at_block(base + (uint32_t)row * 512u, b), u);
                scale_out(x, rs, rights[0], lane);
                if (t >= tl.lo && t < tl.hi && (!shared || lane < 8)) {
                    if (shared) {
#pragma unroll
                        for (int j = 0; j < 16; j++)
                            x[j] = __fadd_rn(x[j], v[j]);
                    } else if (a.p.term) {
                        add_term(a.p, a.n_out, tl.f0, t, x, u);
                    }
                    store_out<TY>(a.p, tl.f0, t, x, u);
                }
            }
        }
        cluster_sync();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_before();
    __syncthreads();
    if (gave_up) {
        // nothing may be in flight when the block ends: its last copies and matrix instructions
        if (warp == kWarpB && lane == 0)
            for (uint32_t back = 1; back <= nb && back <= issued; back++)
                bar_drain(full_b((issued - back) % nb), ((issued - back) / nb) & 1);
        if (warp == kWarpMma && !(PAIR && rank == 1)) {
            if (elect())
                commit<PAIR>(drained);
            __syncwarp();
            bar_drain(drained, 0);
        }
        __syncthreads();
    }
    if (PAIR)
        cluster_sync();                    // neither block ends while the other may still reach into it
    if (warp == kDecWarps) {
        fence_after();
        tmem_free_all<PAIR>(tmem);
    }
}

template <int K, bool PAIR, typename TY> exl3_status launch_form(const Args &a, unsigned grid, unsigned cluster, cudaStream_t s) {
    static_assert(kSmem <= 227 * 1024 - 1536, "shared memory of one block");
    cudaError_t e = allow_smem((const void *)product_kernel<K, PAIR, TY>, kSmem);
    if (e != cudaSuccess)
        return cuda_check(e, "cudaFuncSetAttribute(coded product)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreadsP);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, product_kernel<K, PAIR, TY>, a);
    if (e != cudaSuccess)
        return cuda_check(e, "coded product launch");
    note_launch();
    return cuda_check(cudaGetLastError(), "coded product launch");
}

template <bool PAIR, typename TY> exl3_status launch_k(const Args &a, unsigned grid, unsigned cluster, cudaStream_t s) {
    switch (a.p.K) {
    case 1: return launch_form<1, PAIR, TY>(a, grid, cluster, s);
    case 2: return launch_form<2, PAIR, TY>(a, grid, cluster, s);
    case 3: return launch_form<3, PAIR, TY>(a, grid, cluster, s);
    default: return launch_form<4, PAIR, TY>(a, grid, cluster, s);
    }
}
template <bool PAIR> exl3_status launch_t(const Args &a, unsigned grid, unsigned cluster, cudaStream_t s) {
    return a.p.dt == EXL3_BF16 ? launch_k<PAIR, __nv_bfloat16>(a, grid, cluster, s)
                               : launch_k<PAIR, __half>(a, grid, cluster, s);
}

// token tiles, at most: experts' sizes are not known to the host
int64_t token_tiles(const ProductLaunch &p, int tile_n) {
    const int64_t used = p.T < p.E ? p.T : p.E;
    return p.offsets ? used + (p.T + 7 * used) / tile_n + 1 : (p.T + tile_n - 1) / tile_n;
}

// B stages of `rows` tokens: several steps to a stage when a step is small, so
// that a wait and an arrival serve all of them
void set_b(Args &a, int rows) {
    a.b_steps = rows <= 64 ? 4 : rows <= 128 ? 2 : 1;
    a.b_stages = (int)(kBArea / ((unsigned)(rows * 128) * a.b_steps));
    a.b_stages = a.b_stages > kBStages ? kBStages : a.b_stages;
}

}  // namespace

exl3_status launch_product(const ProductLaunch &p, cudaStream_t s) {
    Args a;
    a.p = p;
    a.n_in = (int)(p.transposed ? p.cols : p.rows);
    a.n_out = (int)(p.transposed ? p.rows : p.cols);
    const int64_t sms = device_sm_count(), pairs = sms / 2;
    const int nf = a.n_out / 128, np = (nf + 1) / 2, steps = a.n_in / kStep;

    // Alone: token tiles of even size, at most kN; blocks that would idle share the sums
    // of the tiles, at least 4 steps each.
    const int64_t n = (p.T + kN - 1) / kN;
    a.tile_n = p.offsets ? (p.T > 16 ? kN : 32) : (int)(((p.T + n - 1) / n + 15) / 16 * 16);
    const int64_t tiles = token_tiles(p, a.tile_n) * nf;
    a.split = 1;
    while (a.split < 8 && tiles * a.split * 2 <= sms && steps >= a.split * 2 * 4)
        a.split *= 2;

    // In pairs, with tiles of up to 512 tokens.  Both forms are estimated in cycles, as
    // measured: a step takes about 1000 (shared memory and the handovers bound it; from
    // 480 columns of a pair on its products do), the results of 64 columns 3000, which
    // pass behind the next tile's sums unless that needs both accumulators.  (333 tokens,
    // 4096 x 12288: 70 us alone in two rounds, 48 in pairs; 4096 tokens of 4096 x 4096 in
    // tiles of 480: 116 us, of 256: 153.)  The experts' tokens are not known here: pairs
    // when an expert has more than 512 on average.  (Pairs / alone, us with the rotation: 16
    // experts 2048 -> 1024, K = 2, of 256 rows each 40.5 / 39.6, 400: 52.7 / 60.7, 600: 80.8 /
    // 86.3, 1024: 115 / 124; skewed, 400 on average 81.9 / 63.2, 600: 93.7 / 88.6, 1024: 132 /
    // 125.  8 experts 4096 -> 4096, K = 4, 400 each 115 / 155, 600: 206 / 219, 1024: 254 / 287;
    // skewed, 400: 146 / 158, 600: 177 / 203, 1024: 292 / 317.  Below 256 alone is ahead, from
    // there to 512 it goes by the rounds, which the host does not know.)
    int pair_n = 0;
    if (p.offsets) {
        pair_n = p.T > 512 * (int64_t)p.E ? 512 : 0;
    } else if (p.T > kN) {
        auto rounds = [](int64_t work, int64_t at_once) { return (work + at_once - 1) / at_once; };
        int64_t best = (a.split > 1 ? 1 : rounds(tiles, sms)) * (steps / a.split) * 1000 + a.tile_n / 64 * 3000;
        for (int t = 512; t >= 256; t -= 32) {
            const int64_t step = t > 480 ? 1000 * t / 480 : 1000, out = t * 3000 / 64;
            const int64_t r = rounds(token_tiles(p, t) * np, pairs);
            const int64_t c = t > kN ? r * (steps * step + out) : r * steps * step + out;
            if (c <= best)
                best = c, pair_n = t;
        }
    }
    if (pair_n) {
        a.tile_n = pair_n;
        a.b_steps = 1;                     // (block 1's decode warps count stages as steps)
        a.b_stages = (int)(kBArea / (a.tile_n * 64u));
        a.b_stages = a.b_stages > kBStages ? kBStages : a.b_stages;
        a.split = 1;
        const int64_t t = token_tiles(p, a.tile_n) * np;
        return launch_t<true>(a, (unsigned)(2 * (t < pairs ? t : pairs)), 2, s);
    }
    set_b(a, a.tile_n);
    const unsigned grid = (unsigned)(a.split > 1 ? tiles * a.split : tiles < sms ? tiles : sms);
    return launch_t<false>(a, grid, (unsigned)a.split, s);
}

exl3_status product_take_wait_timeouts(unsigned int *n) {
    *n = 0;
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_product_timeouts, sizeof v);
    if (e == cudaSuccess && v != 0)
        e = cudaMemcpyToSymbol(g_product_timeouts, &zero, sizeof zero);
    if (e != cudaSuccess)
        return cuda_check(e, "wait timeout count");
    const exl3_status st = few_take_wait_timeouts(n);
    *n += v;
    return st;
}

}  // namespace exl3
