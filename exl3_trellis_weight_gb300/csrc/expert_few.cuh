// expert_few.cuh -- the sums of an expert's few rows with coded matrices, as in
// linear_few.cu: a warp owns 16 outputs, its tiles of codes arrive in a ring and become
// A fragments, the rotated activations lie in shared memory.
//
// The work is a list of steps: for each tile of rows, for each 128 outputs, each 128 inputs.
// How many there are the host does not know (it goes by the picks), and the decoding that
// bounds them cannot be shared, so the blocks - two to an SM, all there at once - take even
// shares of the list, whatever it holds.  A tile's outputs that two blocks share are joined
// in memory: each writes its sums, and the one that is last to come adds them in the order
// of the list.  Codes and activations are asked for steps ahead, across the tiles, and what
// the end of a tile needs at its beginning.
#pragma once

#include "layer.cuh"
#include "linear_few.cuh"

namespace exl3 {

constexpr int kExpertWarps = 16, kExpertThreads = kExpertWarps * 32;

struct ExpertSteps {
    const int4 *tiles;        // expert, first row, rows
    const int32_t *n_tiles;
    int max_tiles;
    int nf, steps;            // 128 outputs and 128 inputs to a tile
    float *part;              // [2 blocks][2][tile_n][128]: sums of tiles that blocks share
    int32_t *done;            // [tiles][nf]: steps of it that are finished
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

// A warp's codes, GROUPS groups of four tiles a step (of the two that a step has), 16 tiles
// ahead.  `left` groups follow at `src`, a step's `stride` bytes apart; then `next` is asked
// for another run of them.
template <int K, int GROUPS> struct CodeRing {
    static constexpr int kLanes = 2 * K, kAtOnce = 4;         // lanes of a tile; tiles of a copy group
    static constexpr int kAhead = kTilesAhead / kAtOnce;      // groups
    static constexpr uint32_t kGroup = kAtOnce * 32 * K, kBytes = kAhead * kGroup;   // of a warp
    static_assert(kLanes * kAtOnce <= 32 && kTilesAhead % kAtOnce == 0, "one copy group is one instruction");
    uint32_t dst;             // of the next group
    int left;
    const char *src;

    template <typename Run> __device__ __forceinline__ void next(uint32_t end, int64_t stride, bool mine, Run run) {
        if (left == 0)
            run(*this);
        if (mine && left > 0)
            tc::copy16(dst, src);
        tc::copy_group();
        src += stride;
        left--;
        dst += kGroup;
        if (dst >= end)
            dst -= kBytes;
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

// TWO: the warps' halves have a matrix each and all inputs of a step (gate and up), and the
// halves' sums stay apart; otherwise each has half of a step's inputs, under the rows' scales
// of that step, and the sums are added.
template <int K, int NB, bool TWO> struct ExpertForm {
    using Ring = CodeRing<K, TWO ? 2 : 1>;
    // inputs of a step: [matrix][64 inputs][NB * 8 rows], and the rows' scales
    static constexpr uint32_t kInputs = (TWO ? 2u : 1u) * 2u * NB * 1024u, kScales = TWO ? 0u : 256u, kZ = kInputs + kScales;
    static constexpr int kStages = NB == 4 && TWO ? (K == 4 ? 2 : 3) : NB == 4 || TWO ? 4 : 6;
    static constexpr uint32_t kRings = kExpertWarps * Ring::kBytes, kSums = 2u * NB * 8u * 512u;
    static constexpr uint32_t kRingAt = kStages * kZ, kSumsAt = kRingAt + kRings;
    static constexpr uint32_t kSmem = kSumsAt + kSums + 1024u;
    static_assert(kSmem <= 106 * 1024 && NB * 32 <= 256, "two blocks an SM, beside 6 KB of other variables");
};

constexpr int kTable = 256;                // tiles that a block keeps the places of

// One block's share of the list.  `op` has
//   codes(half, e, f0): the first code of expert e's outputs f0 on
//   load(to, bar, row0, k, rows, lane): a warp's copies of a step's inputs, bytes(rows) in all
//   fetch(tid, e, row0, rows, f0): a thread's part of the 512 numbers that finish() needs
//   finish(x0, x1, kept, row0, r, f0, lane): a row's sums of both halves, by a warp
template <int K, bool TR, int NB, bool TWO, typename Op>
__device__ __forceinline__ void run_share(const ExpertSteps &p, const Op &op, unsigned int *count) {
    using namespace tc;
    using F = ExpertForm<K, NB, TWO>;
    using Ring = typename F::Ring;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[2 * F::kStages];
    __shared__ int4 table[kTable];
    __shared__ float kept[kExpertThreads];
    __shared__ int gave_up, issued, last;
    __shared__ int ahead[6];               // the next copies of inputs: share's step, its tile of outputs, step; rows
    const uint32_t base = (saddr(smem_raw) + 1023u) & ~1023u;
    unsigned char *const sb = smem_raw + (base - saddr(smem_raw));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int fw = warp & 7, half = warp >> 3, blocks = (int)gridDim.x, block = (int)blockIdx.x;
    const uint32_t bar0 = saddr(bars);
    auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(F::kStages + s); };
    // (the plan is complete: the launch before this one waited for it)
    const int nf = p.nf, steps = p.steps;
    const int n_tiles = __ldcg(p.n_tiles);
    if (tid < kTable && tid < p.max_tiles)
        table[tid] = __ldcg(p.tiles + tid);
    if (tid == 0) {
        for (int s = 0; s < F::kStages; s++) {
            bar_init(full(s), 1);
            bar_init(empty(s), kExpertWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        gave_up = issued = 0;
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
    auto tile_of = [&](int it) { return table[it / nf - first]; };

    // this warp's codes
    const uint32_t ring0 = base + F::kRingAt + (uint32_t)warp * Ring::kBytes, ring1 = ring0 + Ring::kBytes;
    const uint32_t lane16 = (uint32_t)lane * 16;
    const bool mine = lane < Ring::kLanes * Ring::kAtOnce;
    const int64_t along = (int64_t)fw * op.hop_f + (int64_t)((TWO ? 0 : half) * 4 + lane / Ring::kLanes) * op.hop + (lane % Ring::kLanes) * 16;
    const int64_t stride = (TWO ? 4 : 8) * op.hop;
    int ring_it = it0, ring_w = w0;        // where the next run begins
    auto run = [&](Ring &r) {
        const int k = ring_w - ring_it * steps, c = min(steps - k, w0 + n - ring_w);
        if (c > 0) {
            r.src = op.codes(half, tile_of(ring_it).x, ring_it % nf * 128) + along + (int64_t)k * 8 * op.hop;
            r.left = c * (TWO ? 2 : 1);
            ring_w += c;
            ring_it++;
        }
    };
    Ring ring;
    ring.dst = ring0 + lane16;
    ring.left = 0;
    ring.src = nullptr;
#pragma unroll 1
    for (int i = 0; i < Ring::kAhead; i++)
        ring.next(ring1, stride, mine, run);
    if (tid == 0) {
        ahead[0] = 0;
        ahead[1] = it0;
        ahead[2] = w0 - it0 * steps;
        ahead[3] = tile_of(it0).y;
        ahead[4] = (tile_of(it0).z + 7) & ~7;
    }
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // inputs of the next step to stage s, by warp 0
    auto issue = [&](int s) {
        const int k = ahead[2], row0 = ahead[3], rows = ahead[4];
        if (lane == 0)
            bar_expect(full(s), op.bytes(rows));
        __syncwarp();
        op.load(base + (uint32_t)s * F::kZ, full(s), row0, k, rows, lane);
        if (lane == 0) {
            issued = ++ahead[0];
            if (k + 1 < steps) {
                ahead[2] = k + 1;
            } else if (issued < n) {
                const int4 t = tile_of(++ahead[1]);
                ahead[2] = 0;
                ahead[3] = t.y;
                ahead[4] = (t.z + 7) & ~7;
            }
        }
        __syncwarp();
    };
    if (warp == 0)
        for (int i = 0; i < F::kStages && i < n; i++)
            issue(i);
    const Lane l = lane_of<K, TR>(lane >> 2, lane & 3);
    const uint32_t z_mine = base + lane_inputs(lane) + (TWO ? (uint32_t)half * 2u : (uint32_t)half) * (NB * 1024u);
    Words codes(ring0, l);
    int turn = Ring::kAhead;               // groups up to the ring's end
    float *const sums = reinterpret_cast<float *>(sb + F::kSumsAt);
    int s = 0, it = it0;
    uint32_t phase = 0;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n; it++) {
        const int k0 = w0 + i - it * steps, c = min(steps - k0, n - i);
        const bool own_first = i == 0;
        const int4 tl = tile_of(it);
        const int rows = tl.z, f0 = it % nf * 128, row_blocks = (rows + 7) / 8;
        const float number = op.fetch(tid, tl.x, tl.y, rows, f0);
        float acc[NB][4];
#pragma unroll
        for (int b = 0; b < NB; b++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                acc[b][j] = 0.0f;
#pragma unroll 1
        for (int end = i + c; i < end; i++) {
            ok = ok && __all_sync(0xffffffffu, bar_wait(full(s), phase, &gave_up, count));
            const uint32_t z = z_mine + (uint32_t)s * F::kZ;
            float step[NB][4];
            if (!TWO) {
#pragma unroll
                for (int b = 0; b < NB; b++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        step[b][j] = 0.0f;
            }
#pragma unroll 1
            for (int g = 0; g < (TWO ? 2 : 1); g++) {
                copy_wait<Ring::kAhead - 1>();
                __syncwarp();
                if (ok)
                    four_tiles<K, TR, NB, 1>(codes, l, z + g * (NB * 1024u), row_blocks, TWO ? acc : step);
                __syncwarp();              // every lane has read the tiles that the next copies replace
                ring.next(ring1, stride, mine, run);
                turn--;
                codes.move(turn ? Ring::kGroup : Ring::kGroup - Ring::kBytes);
                if (turn == 0)
                    turn = Ring::kAhead;
            }
            if (!TWO) {
                const float2 *scale = reinterpret_cast<const float2 *>(sb + (uint32_t)s * F::kZ + F::kInputs) + (lane & 3);
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const float2 f = scale[4 * b];
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        acc[b][j] = __fmaf_rn(step[b][j], j & 1 ? f.y : f.x, acc[b][j]);
                }
            }
            __syncwarp();
            if (lane == 0)
                bar_arrive(empty(s));
            // the stage before this one is empty by now, or nearly
            if (warp == 0 && i > 0 && i - 1 + F::kStages < n) {
                const int before = s == 0 ? F::kStages - 1 : s - 1;
                if (__all_sync(0xffffffffu, bar_wait(empty(before), s == 0 ? phase ^ 1 : phase, &gave_up, count)))
                    issue(before);
            }
            if (++s == F::kStages)
                s = 0, phase ^= 1;
        }
        // the sums meet in shared memory
        kept[tid] = number;
        if (c == steps) {
#pragma unroll
            for (int b = 0; b < NB; b++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int o = sum_output<K, TR>(fw, lane, j);
                    sums[(half * NB * 8 + sum_row(lane, b, j)) * 128 + 4 * out_at(o >> 2) + (o & 3)] = acc[b][j];
                }
        } else {
            // of a share of the inputs: to memory, and the last to come adds all up
            float *part = p.part + (int64_t)(block * 2 + (own_first ? 0 : 1)) * 2 * (NB * 8 * 128);
#pragma unroll
            for (int b = 0; b < NB; b++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (sum_row(lane, b, j) < rows)
                        __stcg(part + (half * NB * 8 + sum_row(lane, b, j)) * 128 + sum_output<K, TR>(fw, lane, j), acc[b][j]);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                last = atomicAdd(p.done + it, c) + c == steps;
                __threadfence();
            }
            __syncthreads();
            if (!last)
                continue;                  // (`last` is written again behind another barrier)
            const int from = it * steps, b_lo = shares.block_of(from), b_hi = shares.block_of(from + steps - 1);
            for (int q = tid; q < 2 * rows * 32; q += kExpertThreads) {
                const int h = q >= rows * 32 ? 1 : 0, r = (q >> 5) - h * rows, f = q & 31;
                const float *at = p.part + (int64_t)((h * NB * 8 + r) * 128 + f * 4);
                float4 sum = {};
#pragma unroll 4
                for (int b = b_lo; b <= b_hi; b++) {
                    const int own = shares.first(b) >= from ? 0 : 1;
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(at + (int64_t)(b * 2 + own) * 2 * (NB * 8 * 128)));
                    sum.x = __fadd_rn(sum.x, v.x), sum.y = __fadd_rn(sum.y, v.y);
                    sum.z = __fadd_rn(sum.z, v.z), sum.w = __fadd_rn(sum.w, v.w);
                }
                reinterpret_cast<float4 *>(sums)[(h * NB * 8 + r) * 32 + out_at(f)] = sum;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int r = warp; r < rows; r += kExpertWarps) {
            const float4 *at = reinterpret_cast<const float4 *>(sums) + r * 32 + out_at(lane);
            op.finish(at[0], at[NB * 8 * 32], kept, tl.y, r, f0, lane);
        }
        __syncthreads();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (gave_up && tid == 0)               // nothing may be in flight when the block ends
        for (int i = max(0, issued - F::kStages); i < issued; i++)
            bar_drain(full(i % F::kStages), (uint32_t)(i / F::kStages) & 1);
}

}  // namespace exl3
