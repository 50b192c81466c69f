// linear_adapt.cu -- low-rank adapters of many requests when there are more than a
// few tokens: the sums with the rank-sided factor (shrink), the way back (expand)
// and the sums of outer products that are the factors' gradients (outer).
//
// A plan sorts the tokens by adapter (in their order inside one) and cuts each
// adapter's into tiles of 32, so that a tile multiplies by one factor; the host
// never learns the sizes.  The products are a few per cent of the coded product's
// and bound by reading the activations once: m16n8k16 instructions from shared
// memory, fed by asynchronous copies of gathered rows, are far from the limit.
//
// h = gain A x is kept in binary32.  Where it becomes an operand again it is split
// into two of the activations' type, the second the rounding error of the first, and
// both are multiplied (one alone cost half as much again in the results' error);
// binary16 gets a power of two first, for each token where a token has its own sums
// (expand: nothing of one token touches another's), for each adapter where its tokens
// are summed up (outer), so that its range does not matter.
#include "linear.cuh"
#include "tc.cuh"

namespace exl3 {

namespace {

using namespace tc;

constexpr int kTile = 32;                  // tokens of a tile
constexpr int kPad = 8;                    // elements behind a shared-memory row: conflict-free fragments

__device__ __forceinline__ int rank_of(const int32_t *ranks, int i, int rank) {
    return ranks ? min(max(ranks[i], 0), rank) : rank;
}

// 16 bytes, or zeros
__device__ __forceinline__ void copy16z(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"((uint64_t)__cvta_generic_to_global(src)),
                 "r"(real ? 16 : 0)
                 : "memory");
}

// eight neighbouring elements of a row to shared memory, asynchronously where the
// rows are aligned
template <bool VEC> __device__ __forceinline__ void row8(uint32_t dst, const uint16_t *src, bool real) {
    if constexpr (VEC) {
        copy16z(dst, src, real);
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
        if (real)
#pragma unroll
            for (int i = 0; i < 4; i++)
                w[i] = (uint32_t)src[2 * i] | (uint32_t)src[2 * i + 1] << 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
    }
}

template <typename TX> __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four 8 x 8 blocks, transposed; lane l names row l % 8 of block l / 8
__device__ __forceinline__ void load_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void load_n(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// the power of two that takes m to [2^14, 2^15), from where binary16 holds values down to
// 2^-29 of m at its full 11 bits; none for bfloat16, whose range is binary32's, nor for an
// infinite m (its results are not numbers anyway)
template <typename TX> __device__ __forceinline__ void operand_scale(float m, float &up, float &down) {
    up = down = 1.0f;
    if (__is_same(TX, __half) && m > 0.0f && m < 3.0e38f) {
        const int e = max((int)(__float_as_uint(m) >> 23) - 127, -100);
        up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        down = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
    }
}

// v and w, each as the sum of two values of the type, `apart` elements apart
template <typename TX> __device__ __forceinline__ void split2(float v, float w, TX *to, int apart) {
    const uint32_t high = pack2<TX>(v, w);
    const float2 f = unpack2<TX>(high);
    *reinterpret_cast<uint32_t *>(to) = high;
    *reinterpret_cast<uint32_t *>(to + apart) = pack2<TX>(__fsub_rn(v, f.x), __fsub_rn(w, f.y));
}

// ---- plan --------------------------------------------------------------------
// grid: 32 adapters a block, one a warp.  perm: tokens by adapter, seg: where each
// adapter's begin, tiles: the adapter, first place in perm and tokens of each tile.
constexpr int kScan = 4096;                // tokens looked at at a time

__global__ void __launch_bounds__(1024) plan_kernel(const AdaptLaunch a) {
    __shared__ int32_t slot[kScan];
    __shared__ int count[kMaxAdapters], tile0[kMaxAdapters], sums[2][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    count[tid] = 0;
    __syncthreads();
    for (int64_t t0 = 0; t0 < a.T; t0 += 4096) {
        int s[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int64_t t = t0 + k * 1024 + tid;
            s[k] = t < a.T ? a.slots[t] : -1;
        }
        // a count for each adapter of a warp's tokens, added once
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const unsigned same = __match_any_sync(0xffffffffu, s[k]);
            if (s[k] >= 0 && s[k] < a.n && lane == __ffs(same) - 1)
                atomicAdd(&count[s[k]], __popc(same));
        }
    }
    __syncthreads();
    // exclusive sums over the adapters, of tokens and of tiles
    const int c = count[tid];
    int own[2] = {c, (c + kTile - 1) / kTile}, sum[2] = {own[0], own[1]};
#pragma unroll
    for (int k = 0; k < 2; k++) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum[k], d);
            sum[k] += lane >= d ? o : 0;
        }
        if (lane == 31)
            sums[k][warp] = sum[k];
    }
    __syncthreads();
    int at[2];
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int s = sums[k][lane];
        int before = lane < warp ? s : 0;
#pragma unroll
        for (int d = 16; d; d >>= 1)
            before += __shfl_xor_sync(0xffffffffu, before, d);
        at[k] = before + sum[k] - own[k];
    }
    if (blockIdx.x == 0 && tid < a.n) {
        a.plan.seg[tid] = at[0];
        a.plan.largest[tid] = a.plan.largest[a.n + tid] = 0u;
        if (tid == a.n - 1) {
            a.plan.seg[a.n] = at[0] + own[0];
            *a.plan.n_tiles = at[1] + own[1];
        }
    }
    count[tid] = at[0];                    // (each thread its own)
    tile0[tid] = at[1];
    __syncthreads();
    const int i = blockIdx.x * 32 + warp;
    int to = i < a.n ? count[i] : 0;
    const int from = to;
    for (int64_t t0 = 0; t0 < a.T; t0 += kScan) {
        const int n = (int)(a.T - t0 < kScan ? a.T - t0 : kScan);
        __syncthreads();
        for (int t = tid; t < kScan; t += 1024)
            slot[t] = t < n ? a.slots[t0 + t] : -1;
        __syncthreads();
        if (i < a.n)
            for (int t = lane; t - lane < n; t += 256) {
                unsigned b[8];
#pragma unroll
                for (int k = 0; k < 8; k++)
                    b[k] = __ballot_sync(0xffffffffu, slot[t + 32 * k] == i);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    if (b[k] >> lane & 1u)
                        a.plan.perm[to + __popc(b[k] & ((1u << lane) - 1u))] = (int32_t)(t0 + t + 32 * k);
                    to += __popc(b[k]);
                }
            }
    }
    if (i < a.n)
        for (int k = lane; from + k * kTile < to; k += 32)
            a.plan.tiles[tile0[i] + k] = make_int4(i, from + k * kTile, min(kTile, to - from - k * kTile), 0);
}

// a tile's adapter and its tokens [lo, lo + n) of perm; false when there is no such tile
__device__ __forceinline__ bool find_tile(const AdaptLaunch &a, int tile, int &i, int &lo, int &n) {
    const int4 t = a.plan.tiles[tile];     // (behind the last one it is not used)
    i = t.x, lo = t.y, n = t.z;
    return tile < *a.plan.n_tiles;
}

// ---- shrink: h[t][r] = gain_i sum_k M_i[r][k] x[t][k] ---------------------------
// A block takes one tile and a share of the sum (the blocks of a cluster split it);
// warp w the tokens 16 (w % 2) .. and two sixteenths of every step of 128.  Bound by the
// hand-over of steps (a fourth stage changed nothing, twice the split cost a third more):
// 4096 tokens of 4096, rank 16: 15 us, 2.2 TB/s of activations read; twice 4096 x 4096,
// rank 64: 31 us.
constexpr int kShrinkStages = 3;
constexpr int kRow = 128 + kPad;

// MB: sixteens of rows at most (4 up to rank 64)
template <typename TX, bool VEC, int MB> __global__ void __launch_bounds__(256, MB == 4 ? 3 : 2) shrink_kernel(const AdaptLaunch a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const AdaptSide &sd = a.side[blockIdx.y];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int rank = (int)(blockIdx.x % a.split);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int i, lo, n;
    if (!find_tile(a, (int)(blockIdx.x / a.split), i, lo, n))
        return;                            // (the whole cluster)
    const int r = rank_of(a.ranks, i, a.rank), R16 = (a.rank + 15) / 16 * 16, mb = (r + 15) / 16;
    const int steps = sd.n / 128, k_lo = steps * rank / a.split, k_hi = steps * (rank + 1) / a.split;
    const uint32_t base = saddr(smem), stage = (uint32_t)(kTile + R16) * kRow * 2;
    const uint16_t *x = reinterpret_cast<const uint16_t *>(sd.x);
    const uint16_t *M = reinterpret_cast<const uint16_t *>(sd.M) + (size_t)i * a.rank * sd.n;
    // copies of a step: tokens tid / 16 and tid / 16 + 16, rows tid / 16 + 16 m of the factor, 8 elements each
    const int row = tid >> 4, c8 = (tid & 15) * 8;
    const uint16_t *xr[2];
#pragma unroll
    for (int b = 0; b < 2; b++)
        xr[b] = x + (int64_t)(row + 16 * b < n ? a.plan.perm[lo + row + 16 * b] : 0) * sd.stride + c8;
    auto load = [&](int k) {
        if (k < k_hi) {
            const uint32_t st = base + (uint32_t)((k - k_lo) % kShrinkStages) * stage;
#pragma unroll
            for (int b = 0; b < 2; b++)
                row8<VEC>(st + (uint32_t)((row + 16 * b) * kRow + c8) * 2, xr[b] + (int64_t)k * 128, row + 16 * b < n);
#pragma unroll
            for (int m = 0; m < MB; m++)
                if (m < mb) {
                    const bool real = row + 16 * m < r;
                    copy16z(st + (uint32_t)((kTile + row + 16 * m) * kRow + c8) * 2,
                            M + (size_t)(real ? row + 16 * m : 0) * sd.n + k * 128 + c8, real);
                }
        }
        copy_group();
    };
#pragma unroll
    for (int s = 0; s < kShrinkStages - 1; s++)
        load(k_lo + s);
    float acc[2 * MB][4];
#pragma unroll
    for (int b = 0; b < 2 * MB; b++)
#pragma unroll
        for (int e = 0; e < 4; e++)
            acc[b][e] = 0.0f;
    // blocks of 8 x 8: tokens (0-7 | 8-15) x inputs (0-7 | 8-15), rows (0-7 | 8-15) x inputs the other way round
    const uint32_t at = (uint32_t)(((warp & 1) * 16 + (lane & 15)) * kRow + (warp >> 1) * 32 + (lane >> 4) * 8) * 2;
    const uint32_t bt = (uint32_t)((kTile + (lane & 7) + (lane >> 4) * 8) * kRow + (warp >> 1) * 32 + (lane & 8)) * 2;
    for (int k = k_lo; k < k_hi; k++) {
        copy_wait<kShrinkStages - 2>();
        __syncthreads();
        load(k + kShrinkStages - 1);
        const uint32_t st = base + (uint32_t)((k - k_lo) % kShrinkStages) * stage;
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
            uint32_t f[4];
            load_n(st + at + h, f);
#pragma unroll
            for (int m = 0; m < MB; m++)
                if (m < mb) {
                    uint32_t b[4];
                    load_n(st + bt + h + m * 32 * kRow, b);
                    mma<TX>(acc[2 * m], f, b[0], b[1]);
                    mma<TX>(acc[2 * m + 1], f, b[2], b[3]);
                }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // partial sums [4][token][R16] meet in shared memory
    float *const part = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int b = 0; b < 2 * MB; b++)
        if (b < 2 * mb)
#pragma unroll
            for (int e = 0; e < 4; e += 2)
                *reinterpret_cast<float2 *>(part + ((warp >> 1) * kTile + (warp & 1) * 16 + g + 4 * e) * R16 + b * 8 + 2 * j) =
                    make_float2(acc[b][e], acc[b][e + 1]);
    if (a.split > 1)
        cluster_sync();
    else
        __syncthreads();
    const float gain = a.gain[i];
    float m = 0.0f;
    for (int e = tid; e < kTile * a.rank; e += 256) {
        const int t = e / a.rank, q = e % a.rank;
        if (t % a.split != rank || t >= n)
            continue;
        float s = 0.0f;
        if (q < r) {
            for (int b = 0; b < a.split; b++) {
                const uint32_t from = at_block(base + (uint32_t)(t * R16 + q) * 4u, b);
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    float v;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(from + (uint32_t)(w * kTile * R16) * 4u) : "memory");
                    s = __fadd_rn(s, v);
                }
            }
            s = __fmul_rn(s, gain);
        }
        sd.h[(int64_t)a.plan.perm[lo + t] * a.rank + q] = s;
        m = fmaxf(m, fabsf(s));
    }
#pragma unroll
    for (int d = 16; d; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0 && m > 0.0f)
        atomicMax(sd.largest + i, __float_as_uint(m));   // a maximum: any order gives the same
    if (a.split > 1)
        cluster_sync();
}

// ---- expand: term[t] = sum_r h[t][r] M_i[r], which the coded product adds to its own --
// (in binary32: rounded to the results' type it would leave that rounding where it cancels
// the coded part, and a binary16 term can be out of range where the sum is not.  It costs
// what it moves: 4096 tokens forward take 176 us so, 161 with the term in 16 bits in y.)
// A block takes one tile and 512 outputs, 128 at a time; warp w the tokens 16 (w % 2) ..
// and 32 of the outputs, whose sums go out in whole 32-byte sectors as they stand in the
// registers.  Bound by these stores: 4096 x 4096, rank 16: 19 us, 3.4 TB/s written.
template <typename TX> __global__ void __launch_bounds__(256) expand_kernel(const AdaptLaunch a, float *term) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float downs[kTile];
    const AdaptSide &sd = a.side[0];       // h and its way back: M is [rank][n], n outputs
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int i, lo, n;
    if (!find_tile(a, (int)blockIdx.x, i, lo, n))
        return;
    const int r = rank_of(a.ranks, i, a.rank), R16 = (a.rank + 15) / 16 * 16, kb = (r + 15) / 16;
    constexpr int kF = 128 + kPad;
    const int hrow = R16 + kPad;
    TX *const sh = reinterpret_cast<TX *>(smem);                                 // h, twice [32][R16]
    const uint32_t hlow = (uint32_t)(kTile * hrow) * 2;                          // bytes to the second
    const uint32_t sB = saddr(smem) + 2 * hlow, bbytes = (uint32_t)(R16 * kF) * 2;   // two [R16][128]
    const uint16_t *M = reinterpret_cast<const uint16_t *>(sd.M) + (size_t)i * a.rank * sd.n;
    const int f_lo = blockIdx.y * 512, f_hi = min(f_lo + 512, sd.n);
    auto load = [&](int f0, int buf) {
        if (f0 < f_hi)
            for (int e = tid; e < kb * 16 * 16; e += 256) {
                const int q = e >> 4, c = (e & 15) * 8;
                copy16z(sB + buf * bbytes + (uint32_t)(q * kF + c) * 2, M + (size_t)min(q, a.rank - 1) * sd.n + f0 + c, q < r);
            }
        copy_group();
    };
    load(f_lo, 0);
    // h of the tile in the operand's type, each token under its power of two: token tid / 8,
    // elements 2 (tid % 8) + 16 q and the next
    float hv[16], m = 0.0f;
    {
        const int t = tid >> 3, hq = 2 * (tid & 7);
        const float *from = sd.h + (t < n ? (int64_t)a.plan.perm[lo + t] * a.rank : 0);
#pragma unroll
        for (int q = 0; q < 16; q++) {
            const int at = hq + 16 * (q >> 1) + (q & 1);
            hv[q] = t < n && at < r ? from[at] : 0.0f;
            m = fmaxf(m, fabsf(hv[q]));
        }
    }
#pragma unroll
    for (int d = 4; d; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float up, down;
    operand_scale<TX>(m, up, down);
    if ((tid & 7) == 0)
        downs[tid >> 3] = down;            // (read behind the barriers of the first outputs)
#pragma unroll
    for (int q = 0; q < 8; q++)
        if (q < kb)
            split2<TX>(__fmul_rn(hv[2 * q], up), __fmul_rn(hv[2 * q + 1], up), sh + (tid >> 3) * hrow + 2 * (tid & 7) + 16 * q,
                       kTile * hrow);
    const uint32_t ha = saddr(smem) + (uint32_t)(((warp & 1) * 16 + (lane & 15)) * hrow + (lane >> 4) * 8) * 2;
    const uint32_t ba = sB + (uint32_t)((lane & 15) * kF + (warp >> 1) * 32 + (lane >> 4) * 8) * 2;
    // results: tokens 16 (w % 2) + g and 8 on, outputs 32 (w / 2) + 2 j .. of each eight
    float *to[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int t = (warp & 1) * 16 + g + 8 * h;
        to[h] = t < n ? term + (int64_t)a.plan.perm[lo + t] * sd.n + (warp >> 1) * 32 + 2 * j : nullptr;
    }
    for (int f0 = f_lo, buf = 0; f0 < f_hi; f0 += 128, buf ^= 1) {
        copy_wait<0>();
        __syncthreads();                   // (the other buffer is read, too)
        load(f0 + 128, buf ^ 1);
        float acc[4][4];
#pragma unroll
        for (int b = 0; b < 4; b++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[b][e] = 0.0f;
        for (int k = 0; k < kb; k++) {
            uint32_t f[4], f2[4];
            load_n(ha + k * 32, f);
            load_n(ha + k * 32 + hlow, f2);
#pragma unroll
            for (int b = 0; b < 2; b++) {
                uint32_t t[4];
                load_t(ba + buf * bbytes + (uint32_t)(k * 16 * kF + b * 16) * 2, t);
                mma<TX>(acc[2 * b], f, t[0], t[1]);
                mma<TX>(acc[2 * b + 1], f, t[2], t[3]);
                mma<TX>(acc[2 * b], f2, t[0], t[1]);
                mma<TX>(acc[2 * b + 1], f2, t[2], t[3]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (!to[h])
                continue;
            const float d = downs[(warp & 1) * 16 + g + 8 * h];
#pragma unroll
            for (int b = 0; b < 4; b++)
                *reinterpret_cast<float2 *>(to[h] + f0 + 8 * b) = make_float2(__fmul_rn(acc[b][2 * h], d), __fmul_rn(acc[b][2 * h + 1], d));
        }
    }
}

// ---- outer: dM_i[r][k] = sum_{t of i} h[t][r] x[t][k] ------------------------------
// A block takes one adapter, 128 of k (16 a warp) and a share of the adapter's tokens
// (the blocks of a cluster take turns at its tiles of 32).  Bound by latency (a tile is
// 8 KB of x and a hundred instructions a warp between two barriers) and by the adapter
// with the most tokens: blocks in flight count.  Room for rank 64 only, where that is
// enough, lets three blocks share a SM instead of two; with twice the split, 4096 tokens
// x (4096 + 4096), four adapters of rank 64, take 38 us instead of 60, 1001 tokens 8
// instead of 14 (twice the split again: 47 and 13).
constexpr int kOuterStages = 4;
constexpr int kXRow = 128 + kPad;

// It needs nothing of the coded product before it and starts on the SMs that the product
// leaves (1001 tokens in all: 70 us instead of 79; where the product fills the GPU it
// makes no difference): the product lets it go once its own wait has passed, so that h and the plan are
// complete (and are read past L1, which a kernel that has not waited may find stale).
// MB: sixteens of rows at most (4 up to rank 64: fewer registers, three blocks a SM)
template <typename TX, bool VEC, int MB> __global__ void __launch_bounds__(256, MB == 4 ? 3 : 2) outer_kernel(const AdaptLaunch a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int rank = (int)(blockIdx.x % a.split), i = blockIdx.y;
    int chunk = (int)(blockIdx.x / a.split);
    const int side = chunk < a.side[0].n / 128 ? 0 : 1;
    chunk -= side ? a.side[0].n / 128 : 0;
    const AdaptSide &sd = a.side[side];
    const int r = rank_of(a.ranks, i, a.rank), R16 = (a.rank + 15) / 16 * 16, mb = (r + 15) / 16;
    const int lo = __ldcg(a.plan.seg + i), n = __ldcg(a.plan.seg + i + 1) - lo;
    const int hrow = R16 + kPad;
    const uint32_t base = saddr(smem), xbytes = kTile * kXRow * 2, hlow = (uint32_t)(kTile * hrow) * 2, hbytes = 2 * hlow;
    const uint32_t hbase = base + kOuterStages * xbytes;
    float up, down;
    operand_scale<TX>(__uint_as_float(__ldcg(sd.largest + i)), up, down);
    const int tiles = (n + kTile - 1) / kTile;
    const int mine = r > 0 && tiles > rank ? (tiles - 1 - rank) / a.split + 1 : 0;
    const uint16_t *x = reinterpret_cast<const uint16_t *>(sd.x) + chunk * 128;
    // copies of a tile: tokens tid / 16 and tid / 16 + 16, 8 elements each.  The tokens'
    // rows are looked up a tile before they are copied.
    const int row = tid >> 4, c8 = (tid & 15) * 8;
    int next[2];
    auto lookup = [&](int s) {
#pragma unroll
        for (int b = 0; b < 2; b++) {
            const int t = (rank + s * a.split) * kTile + row + 16 * b;
            next[b] = s < mine && t < n ? __ldcg(a.plan.perm + lo + t) : -1;
        }
    };
    auto load = [&](int s) {
        if (s < mine)
#pragma unroll
            for (int b = 0; b < 2; b++)
                row8<VEC>(base + (uint32_t)(s % kOuterStages) * xbytes + (uint32_t)((row + 16 * b) * kXRow + c8) * 2,
                          x + (int64_t)max(next[b], 0) * sd.stride + c8, next[b] >= 0);
        copy_group();
        lookup(s + 1);
    };
    // h of a tile: token tid / 8, elements 2 (tid % 8) + 16 q and the next, in the same way
    const int ht = tid >> 3, hq = 2 * (tid & 7);
    const bool pairs = a.rank % 2 == 0;
    float hv[2 * MB];
    int hnext;
    auto hlookup = [&](int s) {
        const int t = (rank + s * a.split) * kTile + ht;
        hnext = s < mine && t < n ? __ldcg(a.plan.perm + lo + t) : -1;
    };
    auto fetch = [&](int s) {
        const float *from = sd.h + (int64_t)max(hnext, 0) * a.rank;
#pragma unroll
        for (int q = 0; q < MB; q++) {
            const int at = hq + 16 * q;
            if (pairs) {                   // (rows behind r hold zeros)
                const float2 f = hnext >= 0 && at < r ? __ldcg(reinterpret_cast<const float2 *>(from + at)) : make_float2(0.0f, 0.0f);
                hv[2 * q] = f.x, hv[2 * q + 1] = f.y;
            } else {
                hv[2 * q] = hnext >= 0 && at < r ? __ldcg(from + at) : 0.0f;
                hv[2 * q + 1] = hnext >= 0 && at + 1 < r ? __ldcg(from + at + 1) : 0.0f;
            }
        }
        hlookup(s + 1);
    };
    hlookup(0);
    lookup(0);
    fetch(0);
#pragma unroll
    for (int s = 0; s < kOuterStages - 1; s++)
        load(s);
    float acc[MB][2][4];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int b = 0; b < 2; b++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[m][b][e] = 0.0f;
    for (int s = 0; s < mine; s++) {
        TX *const sh = reinterpret_cast<TX *>(smem + kOuterStages * xbytes + (s & 1) * hbytes);
#pragma unroll
        for (int q = 0; q < MB; q++)
            if (q < mb)
                split2<TX>(__fmul_rn(hv[2 * q], up), __fmul_rn(hv[2 * q + 1], up), sh + ht * hrow + hq + 16 * q, kTile * hrow);
        copy_wait<kOuterStages - 2>();
        __syncthreads();
        load(s + kOuterStages - 1);
        fetch(s + 1);
        const uint32_t xs = base + (uint32_t)(s % kOuterStages) * xbytes, hs = hbase + (s & 1) * hbytes;
#pragma unroll
        for (int k = 0; k < kTile / 16; k++) {
            uint32_t b[4];
            load_t(xs + (uint32_t)((k * 16 + (lane & 15)) * kXRow + warp * 16 + (lane >> 4) * 8) * 2, b);
#pragma unroll
            for (int m = 0; m < MB; m++)
                if (m < mb) {
                    uint32_t f[4];         // blocks (tokens 0-7 | 8-15) x (rows 0-7 | 8-15): rows first
                    const uint32_t at = hs + (uint32_t)((k * 16 + (lane & 7) + (lane >> 4) * 8) * hrow + m * 16 + ((lane >> 3) & 1) * 8) * 2;
                    load_t(at, f);
                    mma<TX>(acc[m][0], f, b[0], b[1]);
                    mma<TX>(acc[m][1], f, b[2], b[3]);
                    load_t(at + hlow, f);
                    mma<TX>(acc[m][0], f, b[0], b[1]);
                    mma<TX>(acc[m][1], f, b[2], b[3]);
                }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // partial sums [R16][128] meet in shared memory; block `rank` finishes rows rank, rank + split, ...
    float *const part = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int m = 0; m < MB; m++)
        if (m < mb)
#pragma unroll
            for (int b = 0; b < 2; b++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    part[(m * 16 + g + 8 * (e >> 1)) * 132 + warp * 16 + b * 8 + 2 * j + (e & 1)] = acc[m][b][e];
    if (a.split > 1)
        cluster_sync();
    else
        __syncthreads();
    TX *const out = reinterpret_cast<TX *>(sd.dM) + (size_t)i * a.rank * sd.n + chunk * 128;
    for (int q = rank + (tid >> 5) * a.split; q < a.rank; q += 8 * a.split) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (q < r)
            for (int b = 0; b < a.split; b++) {
                float4 f;
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                             : "r"(at_block(base + (uint32_t)(q * 132 + lane * 4) * 4u, b)) : "memory");
                v[0] = __fadd_rn(v[0], f.x), v[1] = __fadd_rn(v[1], f.y), v[2] = __fadd_rn(v[2], f.z), v[3] = __fadd_rn(v[3], f.w);
            }
        *reinterpret_cast<uint2 *>(out + (size_t)q * sd.n + lane * 4) =
            make_uint2(pack2<TX>(__fmul_rn(v[0], down), __fmul_rn(v[1], down)),
                       pack2<TX>(__fmul_rn(v[2], down), __fmul_rn(v[3], down)));
    }
    if (a.split > 1)
        cluster_sync();
    // the last block to start keeps the grid from ending before the product
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1)
        asm volatile("griddepcontrol.wait;" ::: "memory");
}

// early: the launch may overlap the end of the one before it, whose results the kernel
// waits for (shrink and expand behind the plan, which starts after everything before)
template <typename... P, typename... A>
exl3_status launch(const char *what, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                   bool early, cudaStream_t s, A... args) {
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_smem((const void *)kernel, smem);
        if (e != cudaSuccess)
            return cuda_check(e, what);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = early;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess)
        return cuda_check(e, what);
    note_launch();
    return cuda_check(cudaGetLastError(), what);
}

// rows that are read 16 bytes at a time
bool wide_rows(const AdaptSide &s) { return ((uintptr_t)s.x & 15u) == 0 && s.stride % 8 == 0; }

}  // namespace

size_t adapt_plan_ints(int64_t T, int n) {
    return 4 * ((size_t)T / kTile + n + 1) + (size_t)T + 3 * (size_t)n + 2;
}

AdaptPlan adapt_plan(int32_t *ints, int64_t T, int n) {
    AdaptPlan p;
    p.tiles = reinterpret_cast<int4 *>(ints);
    p.perm = ints + 4 * (T / kTile + n + 1);
    p.seg = p.perm + T;
    p.n_tiles = p.seg + n + 1;
    p.largest = reinterpret_cast<uint32_t *>(p.n_tiles + 1);
    return p;
}

exl3_status launch_adapt_plan(const AdaptLaunch &p, cudaStream_t s) {
    return launch("adapter plan launch", plan_kernel, dim3((unsigned)((p.n + 31) / 32)), 1024, 0, 1, false, s, p);
}

exl3_status launch_shrink(const AdaptLaunch &p0, int sides, cudaStream_t s) {
    AdaptLaunch p = p0;
    const int64_t tiles = p.T / kTile + (p.n < p.T ? p.n : p.T);    // at most
    // blocks that would idle share the sums, at least 4 steps of 128 each
    const int64_t sms = device_sm_count();
    int least = p.side[0].n;
    if (sides > 1 && p.side[1].n < least)
        least = p.side[1].n;
    p.split = 1;
    while (p.split < 8 && tiles * sides * p.split * 2 <= 2 * sms && least / 128 >= p.split * 2 * 4)
        p.split *= 2;
    const int R16 = (p.rank + 15) / 16 * 16;
    const size_t stages = (size_t)kShrinkStages * (kTile + R16) * kRow * 2, part = (size_t)4 * kTile * R16 * 4;
    const size_t smem = stages > part ? stages : part;
    const dim3 grid((unsigned)(tiles * p.split), (unsigned)sides);
    const bool vec = wide_rows(p.side[0]) && (sides < 2 || wide_rows(p.side[1]));
    auto go = [&](auto k) { return launch("adapter shrink launch", k, grid, 256, smem, (unsigned)p.split, true, s, p); };
    if (p.rank > 64) {
        if (p.dt == EXL3_BF16)
            return vec ? go(shrink_kernel<__nv_bfloat16, true, 8>) : go(shrink_kernel<__nv_bfloat16, false, 8>);
        return vec ? go(shrink_kernel<__half, true, 8>) : go(shrink_kernel<__half, false, 8>);
    }
    if (p.dt == EXL3_BF16)
        return vec ? go(shrink_kernel<__nv_bfloat16, true, 4>) : go(shrink_kernel<__nv_bfloat16, false, 4>);
    return vec ? go(shrink_kernel<__half, true, 4>) : go(shrink_kernel<__half, false, 4>);
}

exl3_status launch_expand(const AdaptLaunch &p, float *term, cudaStream_t s) {
    const int64_t tiles = p.T / kTile + (p.n < p.T ? p.n : p.T);
    const int R16 = (p.rank + 15) / 16 * 16;
    const size_t smem = (size_t)2 * kTile * (R16 + kPad) * 2 + (size_t)2 * R16 * (128 + kPad) * 2;
    const dim3 grid((unsigned)tiles, (unsigned)((p.side[0].n + 511) / 512));
    if (p.dt == EXL3_BF16)
        return launch("adapter expand launch", expand_kernel<__nv_bfloat16>, grid, 256, smem, 1, true, s, p, term);
    return launch("adapter expand launch", expand_kernel<__half>, grid, 256, smem, 1, true, s, p, term);
}

exl3_status launch_outer(const AdaptLaunch &p0, cudaStream_t s) {
    AdaptLaunch p = p0;
    // four blocks a SM (they are short) while each has two tiles of an even share
    const int64_t blocks = (int64_t)(p.side[0].n + p.side[1].n) / 128 * p.n, sms = device_sm_count();
    p.split = 1;
    while (p.split < 8 && blocks * p.split * 2 <= 4 * sms && p.T >= (int64_t)p.split * 2 * kTile * p.n)
        p.split *= 2;
    const int R16 = (p.rank + 15) / 16 * 16;
    const size_t stages = (size_t)kOuterStages * kTile * kXRow * 2 + (size_t)4 * kTile * (R16 + kPad) * 2;
    const size_t part = (size_t)R16 * 132 * 4, smem = stages > part ? stages : part;
    const dim3 grid((unsigned)((p.side[0].n + p.side[1].n) / 128 * p.split), (unsigned)p.n);
    const bool vec = wide_rows(p.side[0]) && wide_rows(p.side[1]);
    auto go = [&](auto k) { return launch("adapter gradient launch", k, grid, 256, smem, (unsigned)p.split, p.T > 0, s, p); };
    if (p.rank > 64) {
        if (p.dt == EXL3_BF16)
            return vec ? go(outer_kernel<__nv_bfloat16, true, 8>) : go(outer_kernel<__nv_bfloat16, false, 8>);
        return vec ? go(outer_kernel<__half, true, 8>) : go(outer_kernel<__half, false, 8>);
    }
    if (p.dt == EXL3_BF16)
        return vec ? go(outer_kernel<__nv_bfloat16, true, 4>) : go(outer_kernel<__nv_bfloat16, false, 4>);
    return vec ? go(outer_kernel<__half, true, 4>) : go(outer_kernel<__half, false, 4>);
}

}  // namespace exl3
