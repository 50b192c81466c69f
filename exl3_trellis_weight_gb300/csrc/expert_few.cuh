// expert_few.cuh -- the sums of an expert's few rows with coded matrices, as in
// linear_few.cu: a warp owns 16 outputs, its tiles of codes arrive in a ring and become
// A fragments, the rotated activations lie in shared memory.
//
// The work is a list of steps: for each tile of rows, for each 128 outputs, each 128 inputs.
// How many there are the host does not know (it goes by the picks), and the decoding that
// bounds them cannot be shared, so the blocks - one to an SM, all there at once - take even
// shares of the list, whatever it holds.  A tile's outputs that blocks share are joined in
// memory: each writes its sums, and the one that is last to come adds them in the order of
// the list.  Codes and activations are asked for steps ahead, across the tiles.
//
// A block is four sets of eight warps, and a warp takes 128 inputs of its 16 outputs, eight
// tiles, at a time; which set has which steps is below.  The sets are tied to each other by the
// stages of the inputs.  With two blocks of half the warps to an SM the first was served
// before the second, ended after two thirds of the time and left an SM's issue slots half empty
// (64 tokens over 64 experts, 2048 / 1024, K = 2: 213 us for the layer instead of 190 then);
// 16 warps with all the registers took 232.
#pragma once

#include "expert_form.cuh"
#include "layer.cuh"
#include "linear_few.cuh"

namespace exl3 {

struct ExpertSteps {
    const int4 *tiles;        // expert, first row, rows
    const int32_t *n_tiles;
    int max_tiles;
    int nf, steps;            // 128 outputs and 128 inputs to a tile
    float *part;              // [blocks][2][matrices][rows of a tile][128]: sums of tiles that blocks share
    int32_t *done;            // [tiles][nf]: finished steps of it, of all rows and matrices
};

// `all` steps in even shares: block b begins at step first(b)
struct Shares {
    int each, more;           // the first `more` blocks have one step more
    __device__ __forceinline__ Shares(int all, int blocks) : each(all / blocks), more(all % blocks) {}
    __device__ __forceinline__ int first(int b) const { return b * each + min(b, more); }
    __device__ __forceinline__ int block_of(int step) const {
        const int wide = more * (each + 1);
        return step < wide ? step / (each + 1) : more + (step - wide) / each;     // (each > 0 behind `wide`)
    }
};

// (row g's four inputs of tile i are 8 bytes of chunk 2 i + j / 2 of its row)
__device__ __forceinline__ uint32_t lane_inputs(int lane) {
    const uint32_t g = (uint32_t)lane >> 2, j = (uint32_t)lane & 3u;
    return g * 128u + (((j >> 1) ^ g) << 4) + (j & 1u) * 8u;
}

// places of a warp's sums: output of acc[b][i] within the block's 128, and its row
template <int K, bool TR> __device__ __forceinline__ int sum_output(int fw, int lane, int i) {
    const int g = lane >> 2;
    return fw * 16 + (TR || K <= 2 ? g + 8 * (i >> 1) : 2 * g + (i >> 1));
}
__device__ __forceinline__ int sum_row(int lane, int b, int i) { return b * 8 + 2 * (lane & 3) + (i & 1); }

// ---- a row's 128 outputs, four neighbours to a lane: with few rows a warp to each is the
// shortest way (eight lanes a row took four times as long over the same rows) ------------
__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}
__device__ __forceinline__ float4 mul4(const float4 &a, const float4 &b) {
    return make_float4(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y), __fmul_rn(a.z, b.z), __fmul_rn(a.w, b.w));
}
__device__ __forceinline__ float4 mul4(const float4 &a, float f) { return mul4(a, make_float4(f, f, f, f)); }
// v <- v H
__device__ __forceinline__ float4 rotate_row(float4 v, int lane) {
    const float4 p = make_float4(__fadd_rn(v.x, v.y), __fsub_rn(v.x, v.y), __fadd_rn(v.z, v.w), __fsub_rn(v.z, v.w));
    v = make_float4(__fadd_rn(p.x, p.z), __fadd_rn(p.y, p.w), __fsub_rn(p.x, p.z), __fsub_rn(p.y, p.w));
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) {
        const float sg = (lane & h) ? -1.0f : 1.0f;
        v.x = __fmaf_rn(sg, v.x, __shfl_xor_sync(0xffffffffu, v.x, h));
        v.y = __fmaf_rn(sg, v.y, __shfl_xor_sync(0xffffffffu, v.y, h));
        v.z = __fmaf_rn(sg, v.z, __shfl_xor_sync(0xffffffffu, v.z, h));
        v.w = __fmaf_rn(sg, v.w, __shfl_xor_sync(0xffffffffu, v.w, h));
    }
    return v;
}

// A block's sums in shared memory, [set][row][kSumRow floats]
__device__ __forceinline__ float4 set_sum(const float4 *sums, int set, int every, int rows, int row, int lane) {
    float4 v = sums[(set * rows + row) * (kSumRow / 4) + lane];
    for (set += every; set < kSets; set += every)
        v = add4(v, sums[(set * rows + row) * (kSumRow / 4) + lane]);
    return v;
}

// One more of `all` to have come here; whether it was the last.  (What came before in the
// others' order comes before what the last does next.)
__device__ __forceinline__ uint32_t count_in(uint32_t at, uint32_t all) {
    uint32_t n;
    asm volatile("atom.acq_rel.cta.shared::cta.inc.u32 %0, [%1], %2;" : "=r"(n) : "r"(at), "r"(all - 1) : "memory");
    return n == all - 1;
}

// The same in memory: adds, and returns what was there.  (An atomic between two fences of
// the whole device took longer.)
__device__ __forceinline__ int add_in(int32_t *at, int n) {
    int was;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(was) : "l"(__cvta_generic_to_global(at)), "r"(n) : "memory");
    return was;
}

// tiles that a block keeps the places of: all of them, or those of its share.  There are 1536 at
// most (4096 pairs, 1024 experts), so that a share has part of 13 on 152 SMs, and of 128 on 13.
constexpr int kTable = 128;

// One block's share of the list.  `op` has
//   codes(matrix, e, f0): the first code of expert e's outputs f0 on
//   load(to, bar, row0, k, rows, lane): a warp's copies of a step's inputs, bytes(rows) in all
//   fetch(tid, e, row0, rows, f0): a thread's part of the 512 numbers that finish() needs
//   finish(x0, x1, kept, row0, r, f0, lane): a row's sums (of both matrices), by a warp
template <int K, bool TR, int RB, bool LO, bool TWO, typename Op>
__device__ __forceinline__ void run_share(const ExpertSteps &p, const Op &op, unsigned int *count) {
    using namespace tc;
    using F = ExpertForm<K, RB, LO, TWO>;
    constexpr int G = F::kGroups, M = F::kMatrices, S = F::kStages, L = F::kArrivals, B = F::kMeet;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[L + 2 * B];
    __shared__ uint32_t used[S], filled[L];                    // warps that are done with a stage; times a barrier was armed
    __shared__ int4 table[kTable];
    __shared__ __align__(16) float kept[2][512];
    __shared__ int gave_up;
    __shared__ int4 cursor[G];             // of a group: tile, outputs and step that follow in a stage it is done with
    __shared__ int last[2];                // whether this block joins its first, its other shared tile
    const uint32_t base = (saddr(smem_raw) + 1023u) & ~1023u;
    unsigned char *const sb = smem_raw + (base - saddr(smem_raw));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int fw = warp & 7, set = warp >> 3, matrix = set % M, group = set / M;
    const int blocks = (int)gridDim.x, block = (int)blockIdx.x;
    const uint32_t bar0 = saddr(bars);
    auto full = [&](int b) { return bar0 + 8u * (uint32_t)b; };
    // the sums of a tile are there; have been read
    auto sums_full = [&](int m) { return bar0 + 8u * (uint32_t)(L + m); };
    auto sums_read = [&](int m) { return bar0 + 8u * (uint32_t)(L + B + m); };
    // (the plan is complete: the launch before this one waited for it)
    const int nf = p.nf, steps = p.steps;
    const int n_tiles = __ldcg(p.n_tiles);
    if (tid < kTable && tid < p.max_tiles)
        table[tid] = __ldcg(p.tiles + tid);
    if (tid == 0) {
        for (int b = 0; b < L; b++) {
            bar_init(full(b), 1);
            filled[b] = 0;
        }
        for (int s = 0; s < S; s++)
            used[s] = 0;
        for (int m = 0; m < B; m++) {
            bar_init(sums_full(m), kExpertWarps);
            bar_init(sums_read(m), kExpertWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        gave_up = last[0] = last[1] = 0;
    }
    const int all = n_tiles * nf * steps;
    const Shares shares(all, blocks);
    const int w0 = shares.first(block), n = shares.first(block + 1) - w0;
    if (n == 0) {
        asm volatile("griddepcontrol.wait;" ::: "memory");    // no block ends before what this kernel follows
        return;
    }
    __syncthreads();
    const int it0 = w0 / steps, first = n_tiles > kTable ? it0 / nf : 0;
    if (n_tiles > kTable) {                // this block's tiles only
        if (tid < kTable && first + tid < n_tiles)
            table[tid] = __ldcg(p.tiles + first + tid);
        __syncthreads();
    }
    // the list from the share's first step on: 128 outputs of a tile of rows, and the next ones
    const int tile0 = it0 / nf - first, out0 = it0 % nf, step0 = w0 - it0 * steps;
    auto next_outputs = [&](int &tile, int &out) {
        if (++out == nf)
            out = 0, tile++;
    };

    // this warp's codes: 16 K copies of 16 bytes a step
    const uint32_t ring = base + F::kRingAt + (uint32_t)warp * F::kRing;
    auto chunk = [&](int c) { return (int64_t)(c / (2 * K)) * op.hop + (c % (2 * K)) * 16; };
    const int64_t along = (int64_t)fw * op.hop_f + chunk(lane), stride = 8 * G * op.hop;
    const int more = (int)(chunk(lane + 32) - chunk(lane));
    uint32_t dst = ring + (uint32_t)lane * 16;
    int left = 0, run_i = 0, run_tile = tile0, run_out = out0; // steps left at `src`; where the next run begins
    const char *src = nullptr;
    auto next_codes = [&]() {
        while (left == 0 && run_i < n) {
            const int k = run_i == 0 ? step0 : 0, c = min(steps - k, n - run_i), skip = (group - run_i) & (G - 1);
            if (skip < c) {
                left = (c - skip + G - 1) / G;
                src = op.codes(matrix, table[run_tile].x, run_out * 128) + along + (int64_t)(k + skip) * 8 * op.hop;
            }
            run_i += c;
            next_outputs(run_tile, run_out);
        }
        if (left > 0) {
            if (K > 1 || lane < 16)
                copy16(dst, src);
            if (K == 4 || (K == 3 && lane < 16))
                copy16(dst + 512u, src + more);
            src += stride;
            left--;
        }
        copy_group();
        dst += F::kCodes;
        if (dst >= ring + F::kRing)
            dst -= F::kRing;
    };
#pragma unroll 1
    for (int i = 0; i < F::kAhead; i++)
        next_codes();
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // inputs of step i of the share, which is step k of a tile, by a warp
    auto issue = [&](int i, int tile, int k) {
        const int s = F::stage(i), b = F::arrival(i), rows = (table[tile].z + 7) & ~7;
        if (lane == 0) {
            filled[b]++;
            bar_expect(full(b), op.bytes(rows));
        }
        __syncwarp();
        op.load(base + (uint32_t)s * F::kZ, full(b), table[tile].y, k, rows, lane);
    };
    if (warp < S && warp < n)
        issue(warp, (w0 + warp) / steps / nf - first, (w0 + warp) % steps);
    if (tid < G) {
        const int it = (w0 + S + tid) / steps;
        cursor[tid] = make_int4(it / nf - first, it % nf, w0 + S + tid - it * steps, 0);
    }
    const Lane l = lane_of<K, TR>(lane >> 2, lane & 3);
    const uint32_t z_mine = base + lane_inputs(lane) + (uint32_t)matrix * (2u * F::kPanel);
    Words codes(ring, l);
    int turn = F::kAhead;                  // steps up to the ring's end
    // sums of a shared tile: of the block's first one, or its other
    auto part_of = [&](int b, int which, int m) { return p.part + (int64_t)((b * 2 + which) * M + m) * (F::kRows * 128); };
    __syncthreads();                       // (the cursors)
    bool ok = true;
    int it = it0, tile = tile0, out = out0;
#pragma unroll 1
    for (int i = 0; i < n; it++, next_outputs(tile, out)) {
        const bool own_first = i == 0;
        const int c = min(steps - (own_first ? step0 : 0), n - i), end = i + c;
        const int4 tl = table[tile];
        const int rows = tl.z, f0 = out * 128, row_blocks = (rows + 7) / 8;
        const float number = tid < 512 ? op.fetch(tid, tl.x, tl.y, rows, f0) : 0.0f;
        float acc[RB][4];
#pragma unroll
        for (int b = 0; b < RB; b++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                acc[b][j] = 0.0f;
        i += (group - i) & (G - 1);
#pragma unroll 1
        for (; i < end; i += G) {
            const int s = F::stage(i);
            ok = ok && __all_sync(0xffffffffu, bar_wait(full(F::arrival(i)), F::parity(i), &gave_up, count));
            copy_wait<F::kAhead - 1>();
            __syncwarp();
            if (ok) {
                const uint32_t z0 = z_mine + (uint32_t)s * F::kZ;
                const uint32_t z[4] = {z0, z0 ^ 32u, z0 ^ 64u, z0 ^ 96u};
                if constexpr (TWO) {
                    eight_tiles<K, TR, RB, LO, F::kPanel>(codes, l, z, row_blocks, acc);
                } else {
                    float step[RB][4];
#pragma unroll
                    for (int b = 0; b < RB; b++)
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            step[b][j] = 0.0f;
                    eight_tiles<K, TR, RB, LO, F::kPanel>(codes, l, z, row_blocks, step);
                    const float2 *scale = reinterpret_cast<const float2 *>(sb + (uint32_t)s * F::kZ + F::kInputs) + (lane & 3);
#pragma unroll
                    for (int b = 0; b < RB; b++) {
                        const float2 f = scale[4 * b];
#pragma unroll
                        for (int j = 0; j < 4; j++)
                            acc[b][j] = __fmaf_rn(step[b][j], j & 1 ? f.y : f.x, acc[b][j]);
                    }
                }
            }
            __syncwarp();                  // every lane has read what the next copies replace
            next_codes();
            turn--;
            codes.move(turn ? F::kCodes : F::kCodes - F::kRing);
            if (turn == 0)
                turn = F::kAhead;
            // whoever is the last to be done with a stage asks for its next inputs (a warp that
            // waited for the others instead was the last itself: a quarter of the time)
            if (ok && i + S < n) {
                uint32_t before = 0;
                if (lane == 0)
                    before = count_in(saddr(used + s), kExpertWarps / G);
                if (__shfl_sync(0xffffffffu, before, 0) != 0u) {
                    int4 at = cursor[group];
                    issue(i + S, at.x, at.z);
                    for (at.z += G; at.z >= steps; at.z -= steps)
                        next_outputs(at.x, at.y);
                    __syncwarp();
                    if (lane == 0)
                        cursor[group] = at;
                }
            }
        }
        i = end;
        // the row that this warp finishes, from another set on at each tile
        const int row = (warp + it * 8) % kExpertWarps;
        // the sums meet in shared memory, once the rows of the tile before have been read
        const int m_at = (it - it0) % B;
        const uint32_t m_parity = (uint32_t)((it - it0) / B) & 1;
        float *const sums = reinterpret_cast<float *>(sb + F::kSumsAt + m_at * F::kSums);
        ok = ok && __all_sync(0xffffffffu, bar_wait(sums_read(m_at), m_parity ^ 1, &gave_up, count));
        if (tid < 512)
            kept[m_at][tid] = number;
#pragma unroll
        for (int b = 0; b < RB; b++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                sums[(set * F::kRows + sum_row(lane, b, j)) * kSumRow + sum_output<K, TR>(fw, lane, j)] = acc[b][j];
        __syncwarp();
        if (lane == 0)
            bar_arrive(sums_full(m_at));
        const float4 *const from = reinterpret_cast<const float4 *>(sums);
        if (c == steps) {
            // (a warp without a row goes on)
            if (row < rows) {
                ok = ok && __all_sync(0xffffffffu, bar_wait(sums_full(m_at), m_parity, &gave_up, count));
                if (ok)
                    op.finish(set_sum(from, 0, M, F::kRows, row, lane), TWO ? set_sum(from, 1, M, F::kRows, row, lane) : float4{}, kept[m_at],
                              tl.y, row, f0, lane);
            }
        } else {
            // of a share of the inputs: to memory, a row of a matrix to a warp, and whichever row's
            // last share comes from here says so (no meeting of the block: one to eight tokens
            // gained 1 %)
            if (row < M * rows)
                ok = ok && __all_sync(0xffffffffu, bar_wait(sums_full(m_at), m_parity, &gave_up, count));
#pragma unroll 1
            for (int q = row; q < M * rows; q += kExpertWarps) {
                const int m = q >= rows ? 1 : 0, r = q - m * rows;
                __stcg(reinterpret_cast<float4 *>(part_of(block, own_first ? 0 : 1, m) + r * 128) + lane, set_sum(from, m, M, F::kRows, r, lane));
                __syncwarp();
                if (lane == 0 && add_in(p.done + it, c) + c == steps * M * rows)
                    last[own_first ? 0 : 1] = 1;
            }
        }
        __syncwarp();
        if (lane == 0)
            bar_arrive(sums_read(m_at));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // whose last share came from here, is added up: a row to a warp, both tiles at once where
    // they have rows for half the warps at most
    constexpr int kAtOnce = F::kRows <= kExpertWarps / 2 ? 2 : 1;
#pragma unroll 1
    for (int turn = 0; turn < 2; turn += kAtOnce) {
        if (!last[turn] && !last[turn + kAtOnce - 1])
            continue;
        const int which = kAtOnce == 2 ? warp / (kExpertWarps / 2) : turn, row = kAtOnce == 2 ? warp % (kExpertWarps / 2) : warp;
        const int t = kAtOnce == 2 ? tid & 511 : tid;
        const int at = which ? it - 1 : it0, lo = at * steps, b_lo = shares.block_of(lo), b_hi = shares.block_of(lo + steps - 1);
        const int4 tl = table[at / nf - first];
        const int rows = last[which] ? tl.z : 0, f0 = at % nf * 128;
        const float number = t < 512 && rows ? op.fetch(t, tl.x, tl.y, rows, f0) : 0.0f;
        float4 v[M];
#pragma unroll
        for (int m = 0; m < M; m++)
            v[m] = float4{};
        if (row < rows) {
#pragma unroll 4
            for (int b = b_lo; b <= b_hi; b++)
#pragma unroll
                for (int m = 0; m < M; m++)
                    v[m] = add4(v[m], __ldcg(reinterpret_cast<const float4 *>(part_of(b, shares.first(b) >= lo ? 0 : 1, m) + row * 128) + lane));
        }
        __syncthreads();
        if (t < 512)
            kept[which][t] = number;
        __syncthreads();
        if (row < rows)
            op.finish(v[0], v[M - 1], kept[which], tl.y, row, f0, lane);
    }
    if (gave_up && tid == 0)               // nothing may be in flight when the block ends
        for (int b = 0; b < L; b++)
            if (filled[b])
                bar_drain(full(b), (filled[b] - 1) & 1);
}

}  // namespace exl3
