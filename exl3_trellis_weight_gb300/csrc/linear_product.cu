// linear_product.cu -- y = z V H . right . 2^-7 s (see linear.cuh) with V decoded
// from the codes on the way into the tensor cores.
//
// The product runs transposed: a block owns 128 outputs (the lanes of its
// accumulator) and up to 256 tokens (its columns), so that a weight is decoded
// once for 256 tokens and a single token still fills every lane.  Warps have
// roles:
//   0-7    decode: 32 weights of every 128 x 64 step each, from registers that
//          were loaded kAhead steps before, to a swizzled operand stage.  The
//          weights of a tile row run along the outputs (x W^) or along the sum
//          (x W^^T): the first is stored as an operand whose rows run along M,
//          the second along K, and only the descriptor differs;
//   8-11   results: accumulator -> shared memory (one token per row) -> H over
//          the 128 outputs (16 to a thread) -> scales, adapters, one rounding;
//   12     bulk copies of the rotated activations, one contiguous block a step;
//   13     issues the matrix instructions (128 x N x 16, binary16 in, binary32 out).
// Two accumulators let the results of one tile overlap the sums of the next.
//
// With few tiles (decode), the sum is split over the `split` blocks of a
// cluster; each leaves its partial sums in its shared memory and block r adds
// up, in block order, and finishes tokens r, r + split, ...
//
// Bound by the integer and half-precision pipes of the decode (about 6
// instructions a weight) for few tokens, by the tensor cores and shared memory
// for many.
//
// Every wait is bounded (tc.cuh); after one gives up the block stops issuing,
// waits for what it has in flight, and its results are void (counted in
// exl3_wait_timeouts).
#include "linear.cuh"
#include "tc.cuh"

namespace exl3 {

namespace {

using namespace tc;

constexpr int kDecWarps = 8, kOutWarps = 4;
constexpr int kThreadsP = (kDecWarps + kOutWarps + 2) * 32;
constexpr int kN = 256;                    // tokens of a tile, at most
constexpr int kStep = 64;                  // inputs of a step
constexpr int kStages = 4;
constexpr int kAhead = 4;                  // steps whose codes are in flight
constexpr uint32_t kABytes = 128 * kStep * 2, kBBytes = kN * kStep * 2;
constexpr uint32_t kStageB = kStages * kABytes;             // B stages behind the A stages
constexpr uint32_t kOutOff = kStageB + kStages * kBBytes;   // 32 tokens x 128 outputs, fp32
constexpr uint32_t kSmem = kOutOff + 32 * 128 * 4 + 1024;   // + alignment slack

__device__ unsigned int g_product_timeouts;

// Codebook levels of two windows: fl16(fl32(n c)), n = bytesum - 510.  n is exact
// in binary16 (1024 + bytesum is the half with these bits), and
// fma(n, ch, fl16(n cl)) rounds to the same level for each of the 1021 sums.
constexpr uint32_t kLevelHi = 0x1EED1EEDu;      // ch = 0x1.bb4p-8
constexpr uint32_t kLevelLo = 0x802F802Fu;      // cl = -47 x 2^-24
__device__ __forceinline__ uint32_t levels2(uint32_t s0, uint32_t s1) {
    const uint32_t a = __dp4a(s0 * kMul1Mult, 0x01010101u, 0x6400u);
    const uint32_t b = __dp4a(s1 * kMul1Mult, 0x01010101u, 0x6400u);
    const uint32_t m = __byte_perm(a, b, 0x5410);
    const uint32_t off = 0xE5FEE5FEu;           // -1534
    const __half2 n = __hadd2_rn(*reinterpret_cast<const __half2 *>(&m), *reinterpret_cast<const __half2 *>(&off));
    const uint32_t hi = kLevelHi, lo = kLevelLo;
    const __half2 t = __hmul2_rn(n, *reinterpret_cast<const __half2 *>(&lo));
    const __half2 v = __hfma2(n, *reinterpret_cast<const __half2 *>(&hi), t);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A tile row of 16 weights ends with the last bit of r[NR - 1]; its windows need
// 15 bits before it: 15 + 16 K bits in NR words.
template <int K> struct RowBits { static constexpr int NR = (15 + 16 * K + 31) / 32; };

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

template <int K> __device__ __forceinline__ void load_codes(const uint32_t *p, uint32_t (&w)[K]) {
    if constexpr (K == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (K == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < K; i++)
            w[i] = __ldg(p + i);
    }
}

// 32 weights (two tile rows) of this thread to the operand stage.  Threads of
// odd q store their second row first, so that the eight lanes of a store phase
// cover all banks.
template <int K>
__device__ __forceinline__ void decode32(const uint32_t (&w)[K], int lane, uint32_t first, uint32_t second) {
    constexpr int NR = RowBits<K>::NR;
    const uint32_t prev = __shfl_sync(0xffffffffu, w[K - 1], (lane + 28) & 31);   // the eight q of a tile in a ring
    uint32_t r0[NR], r1[NR];
    if constexpr (K == 1) {
        r0[0] = __funnelshift_r(w[0], prev, 16);
        r1[0] = w[0];
    } else if constexpr (K == 2) {
        r0[0] = prev, r0[1] = w[0];
        r1[0] = w[0], r1[1] = w[1];
    } else if constexpr (K == 3) {
        r0[0] = __funnelshift_r(w[0], prev, 16), r0[1] = __funnelshift_r(w[1], w[0], 16);
        r1[0] = w[1], r1[1] = w[2];
    } else {
        r0[0] = prev, r0[1] = w[0], r0[2] = w[1];
        r1[0] = w[1], r1[1] = w[2], r1[2] = w[3];
    }
    const bool odd = (lane & 4) != 0;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        uint32_t r[NR];
#pragma unroll
        for (int j = 0; j < NR; j++)
            r[j] = (i == 0) == odd ? r1[j] : r0[j];
        const uint32_t at = i ? second : first;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t v[4];
#pragma unroll
            for (int p = 0; p < 4; p++) {
                const int c = 8 * h + 2 * p;
                v[p] = levels2(window<NR>(r, (15 - c) * K), window<NR>(r, (14 - c) * K));
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (h << 4)), "r"(v[0]), "r"(v[1]),
                         "r"(v[2]), "r"(v[3])
                         : "memory");
        }
    }
}

struct Tile {
    int e;            // expert
    int f0;           // first output
    int64_t t0;       // first token column, a multiple of 8 (columns before lo are not stored)
    int64_t lo, hi;   // tokens of the expert inside [t0, t0 + n)
    int n;            // columns, a multiple of 16
};

// Shared list of token tiles: expert e has first[e + 1] - first[e] of them
struct Plan {
    int32_t off[kMaxExperts + 1];
    int32_t first[kMaxExperts + 1];
};

struct Args {
    ProductLaunch p;
    int n_in, n_out;
    int tile_n;          // tokens of a tile (a multiple of 16 up to kN)
    int split;           // blocks of a cluster, each with its share of the steps
};

__device__ __forceinline__ int clamp_off(int32_t v, int64_t T) { return v < 0 ? 0 : (int64_t)v > T ? (int)T : v; }

__device__ __forceinline__ int tiles_of(int lo, int hi, int tile_n) {
    return hi > lo ? (hi - (lo & ~7) + tile_n - 1) / tile_n : 0;
}

// tile `it`: outputs fastest, so that blocks running side by side share their tokens
__device__ __forceinline__ Tile make_tile(const Args &a, const Plan *plan, int64_t it) {
    Tile t;
    const int nf = a.n_out / 128;
    int j = (int)(it / nf);
    t.f0 = (int)(it % nf) * 128;
    int64_t lo = 0, hi = a.p.T;
    t.e = 0;
    if (a.p.offsets) {
        int l = 0, h = a.p.E - 1;        // last e with first[e] <= j
        while (l < h) {
            const int m = (l + h + 1) >> 1;
            if (plan->first[m] <= j)
                l = m;
            else
                h = m - 1;
        }
        t.e = l;
        j -= plan->first[l];
        lo = plan->off[l];
        hi = max(lo, (int64_t)plan->off[l + 1]);
    }
    t.t0 = (lo & ~7ll) + (int64_t)j * a.tile_n;
    t.lo = lo > t.t0 ? lo : t.t0;
    t.hi = hi < t.t0 + a.tile_n ? hi : t.t0 + a.tile_n;
    t.n = (int)((t.hi - t.t0 + 15) / 16 * 16);
    return t;
}

// outputs 4u + 32m + i (m, i < 4) of one token to v[4m + i]: H over the 128, eight threads to a token
__device__ __forceinline__ void rotate_out(float (&v)[16], int lane) {
#pragma unroll
    for (int h = 1; h < 16; h <<= 1)
#pragma unroll
        for (int i = 0; i < 16; i++)
            if ((i & h) == 0) {
                const float p = v[i], q = v[i + h];
                v[i] = __fadd_rn(p, q);
                v[i + h] = __fsub_rn(p, q);
            }
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
        const float sg = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 16; i++)
            v[i] = __fmaf_rn(sg, v[i], __shfl_xor_sync(0xffffffffu, v[i], h));
    }
}

template <typename TY>
__device__ __forceinline__ void finish_token(const Args &a, const Tile &tl, int64_t t, float (&v)[16], int u) {
    const ProductLaunch &p = a.p;
    const float s = __fmul_rn(p.rscale[t], __fmul_rn(p.scale[tl.e], 0x1p-7f));
    const float *right = p.right + (size_t)tl.e * a.n_out + tl.f0 + 4 * u;
#pragma unroll
    for (int m = 0; m < 4; m++) {
        const float4 r = __ldg(reinterpret_cast<const float4 *>(right + 32 * m));
        v[4 * m] = __fmul_rn(__fmul_rn(v[4 * m], s), r.x);
        v[4 * m + 1] = __fmul_rn(__fmul_rn(v[4 * m + 1], s), r.y);
        v[4 * m + 2] = __fmul_rn(__fmul_rn(v[4 * m + 2], s), r.z);
        v[4 * m + 3] = __fmul_rn(__fmul_rn(v[4 * m + 3], s), r.w);
    }
    if (p.B) {
        const int ad = p.slots[t];
        if (ad >= 0 && ad < p.n_adapters) {
            const int r = p.ranks ? min(max(p.ranks[ad], 0), p.rank) : p.rank;
            const TY *b = reinterpret_cast<const TY *>(p.B) + (size_t)ad * p.rank * a.n_out + tl.f0 + 4 * u;
            const float *h = p.h + t * p.rank;
            for (int j = 0; j < r; j++, b += a.n_out) {
                const float hj = h[j];
#pragma unroll
                for (int m = 0; m < 4; m++) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(b + 32 * m));
                    const float2 x = unpack2<TY>(w.x), y = unpack2<TY>(w.y);
                    v[4 * m] = __fmaf_rn(hj, x.x, v[4 * m]);
                    v[4 * m + 1] = __fmaf_rn(hj, x.y, v[4 * m + 1]);
                    v[4 * m + 2] = __fmaf_rn(hj, y.x, v[4 * m + 2]);
                    v[4 * m + 3] = __fmaf_rn(hj, y.y, v[4 * m + 3]);
                }
            }
        }
    }
    TY *y = reinterpret_cast<TY *>(p.y) + t * p.y_stride + tl.f0 + 4 * u;
    if ((((uintptr_t)p.y | (uintptr_t)(p.y_stride * 2)) & 7u) == 0) {
#pragma unroll
        for (int m = 0; m < 4; m++)
            *reinterpret_cast<uint2 *>(y + 32 * m) =
                make_uint2(pack2<TY>(v[4 * m], v[4 * m + 1]), pack2<TY>(v[4 * m + 2], v[4 * m + 3]));
    } else {
#pragma unroll
        for (int m = 0; m < 4; m++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                y[32 * m + i] = from_f32<TY>(v[4 * m + i]);
    }
}

__device__ __forceinline__ void finish(const Args &a, const Tile &tl, int64_t t, float (&v)[16], int lane) {
    rotate_out(v, lane);
    if (t < tl.lo || t >= tl.hi)
        return;
    if (a.p.dt == EXL3_BF16)
        finish_token<__nv_bfloat16>(a, tl, t, v, lane & 7);
    else
        finish_token<__half>(a, tl, t, v, lane & 7);
}

template <int K>
__global__ void __launch_bounds__(kThreadsP, 1) product_kernel(const __grid_constant__ Args a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long bars[3 * kStages + 5];
    __shared__ Plan plan;
    __shared__ uint32_t tmem_at;
    __shared__ int gave_up;
    const uint32_t base = (saddr(smem_raw) + 1023u) & ~1023u;
    unsigned char *const sb = smem_raw + (base - saddr(smem_raw));
    const uint32_t bar0 = saddr(bars);
    auto full_a = [&](int s) { return bar0 + 8u * s; };
    auto full_b = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto empty = [&](int s) { return bar0 + 8u * (2 * kStages + s); };
    auto acc_full = [&](int i) { return bar0 + 8u * (3 * kStages + i); };
    auto acc_empty = [&](int i) { return bar0 + 8u * (3 * kStages + 2 + i); };
    const uint32_t drained = bar0 + 8u * (3 * kStages + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < kStages; s++) {
            bar_init(full_a(s), kDecWarps);
            bar_init(full_b(s), 1);
            bar_init(empty(s), 1);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(acc_full(i), 1);
            bar_init(acc_empty(i), kOutWarps);
        }
        bar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        gave_up = 0;
    }
    if (warp == kDecWarps)
        tmem_alloc<512>(saddr(&tmem_at));
    // token tiles of each expert
    if (a.p.offsets) {
        for (int i = tid; i <= a.p.E; i += kThreadsP)
            plan.off[i] = clamp_off(a.p.offsets[i], a.p.T);
        __syncthreads();
        if (warp == 0) {
            int at = 0;
            for (int e0 = 0; e0 < a.p.E; e0 += 32) {
                const int e = e0 + lane;
                int n = e < a.p.E ? tiles_of(plan.off[e], plan.off[e + 1], a.tile_n) : 0;
                int sum = n;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, sum, d);
                    sum += lane >= d ? o : 0;
                }
                if (e < a.p.E)
                    plan.first[e] = at + sum - n;
                at += __shfl_sync(0xffffffffu, sum, 31);
            }
            if (lane == 0)
                plan.first[a.p.E] = at;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_at;
    const int64_t n_tok = a.p.offsets ? plan.first[a.p.E] : (a.p.T + a.tile_n - 1) / a.tile_n;
    const int64_t n_tiles = n_tok * (a.n_out / 128);
    const int rank = a.split > 1 ? (int)(blockIdx.x % a.split) : 0;
    const int64_t it0 = blockIdx.x / a.split, dit = a.split > 1 ? n_tiles : gridDim.x;   // one tile a cluster
    const int steps = a.n_in / kStep;
    const int k_lo = (int)((int64_t)steps * rank / a.split), k_hi = (int)((int64_t)steps * (rank + 1) / a.split);
    const int64_t NP = act_rows(a.p.T);
    unsigned int *const count = &g_product_timeouts;

    uint32_t issued = 0;                   // bulk copies (of the thread that makes them)
    if (warp < kDecWarps) {
        // ---- decode ----
        const int q = lane >> 2, tc = lane & 3;
        const int64_t tiles_c = a.p.cols / 16;
        // tile of this thread inside a step, and its rows in the operand stage
        const int tr = a.p.transposed ? warp : warp >> 1, tcol = a.p.transposed ? tc : (warp & 1) * 4 + tc;
        const int64_t hop = (a.p.transposed ? 4 : 4 * tiles_c) * (8 * K);
        const uint32_t panel = a.p.transposed ? (uint32_t)warp * 16u * 128u
                                              : (uint32_t)(warp & 1) * 8192u + (uint32_t)(warp >> 1) * 16u * 128u;
        const int odd = q & 1, ra = 2 * q + odd, rb = 2 * q + 1 - odd;
        const uint32_t offa = panel + ra * 128 + (((2 * tc) ^ (ra & 7)) << 4);
        const uint32_t offb = panel + rb * 128 + (((2 * tc) ^ (rb & 7)) << 4);
        uint32_t it_step = 0;
        bool ok = true;
        for (int64_t it = it0; ok && it < n_tiles; it += dit) {
            const Tile tl = make_tile(a, &plan, it);
            const int64_t r0 = a.p.transposed ? tl.f0 / 16 + tr : (int64_t)k_lo * 4 + tr;
            const int64_t c0 = a.p.transposed ? (int64_t)k_lo * 4 + tcol : tl.f0 / 16 + tcol;
            const uint32_t *p = a.p.codes + (size_t)tl.e * (a.p.rows / 16) * tiles_c * (8 * K) +
                                (size_t)(r0 * tiles_c + c0) * (8 * K) + q * K;
            uint32_t w[kAhead][K];
#pragma unroll
            for (int i = 0; i < kAhead; i++)
                if (k_lo + i < k_hi)
                    load_codes<K>(p + i * hop, w[i]);
            for (int k = k_lo; ok && k < k_hi; k += kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; i++) {
                    if (k + i < k_hi && ok) {
                        const int s = it_step % kStages;
                        const uint32_t round = it_step / kStages;
                        if (round && !bar_wait(empty(s), (round - 1) & 1, &gave_up, count))
                            ok = false;
                        // every lane of the warp goes on or none: a lane that gave up takes the others along
                        ok = __all_sync(0xffffffffu, ok);
                        if (ok) {
                            const uint32_t st = base + s * kABytes;
                            decode32<K>(w[i], lane, st + offa, st + offb);
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0)
                                bar_arrive(full_a(s));
                            if (k + i + kAhead < k_hi)
                                load_codes<K>(p + (int64_t)(k + i + kAhead - k_lo) * hop, w[i]);
                            it_step++;
                        }
                    }
                }
            }
        }
    } else if (warp < kDecWarps + kOutWarps) {
        // ---- results ----
        const int ow = warp - kDecWarps;
        float *const buf = reinterpret_cast<float *>(sb + (a.split > 1 ? 0 : kOutOff));
        asm volatile("griddepcontrol.wait;" ::: "memory");
        uint32_t i_acc = 0;
        for (int64_t it = it0; it < n_tiles; it += dit, i_acc++) {
            const Tile tl = make_tile(a, &plan, it);
            const int d = i_acc & 1;
            bool ok = bar_wait(acc_full(d), (i_acc >> 1) & 1, &gave_up, count);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            fence_after();
            for (int c0 = 0; c0 < tl.n; c0 += 32) {
                float v[32];
                tmem_load32(tmem + (uint32_t)(ow * 32) * 65536u + d * kN + c0, v);
                float *const dst = buf + (a.split > 1 ? c0 * 128 : 0) + ow * 32 + lane;
#pragma unroll
                for (int i = 0; i < 32; i++)
                    dst[i * 128] = v[i];
                if (a.split > 1)
                    continue;
                asm volatile("bar.sync 1, 128;" ::: "memory");
                // 16 tokens at a time, eight threads to a token
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    const int row = g * 16 + ow * 4 + (lane >> 3);
                    const float4 *src = reinterpret_cast<const float4 *>(buf + row * 128) + (lane & 7);
                    float x[16];
#pragma unroll
                    for (int m = 0; m < 4; m++) {
                        const float4 f = src[8 * m];
                        x[4 * m] = f.x, x[4 * m + 1] = f.y, x[4 * m + 2] = f.z, x[4 * m + 3] = f.w;
                    }
                    finish(a, tl, tl.t0 + c0 + row, x, lane);
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            fence_before();
            __syncwarp();
            if (lane == 0)
                bar_arrive(acc_empty(d));
        }
    } else if (warp == kDecWarps + kOutWarps) {
        // ---- activations ----
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (lane == 0) {
            uint32_t it_step = 0;
            bool ok = true;
            for (int64_t it = it0; ok && it < n_tiles; it += dit) {
                const Tile tl = make_tile(a, &plan, it);
                const unsigned char *src = a.p.image + ((int64_t)k_lo * NP + tl.t0) * 128;
                for (int k = k_lo; k < k_hi; k++, src += NP * 128) {
                    const int s = it_step % kStages;
                    const uint32_t round = it_step / kStages;
                    if (round && !bar_wait(empty(s), (round - 1) & 1, &gave_up, count)) {
                        ok = false;
                        break;
                    }
                    bar_expect(full_b(s), (uint32_t)tl.n * 128u);
                    bulk_load(base + kStageB + s * kBBytes, src, (uint32_t)tl.n * 128u, full_b(s));
                    it_step++;
                }
            }
            issued = it_step;
        }
    } else {
        // ---- matrix instructions ----
        if (lane == 0) {
            uint32_t it_step = 0, i_acc = 0;
            bool ok = true;
            for (int64_t it = it0; ok && it < n_tiles; it += dit, i_acc++) {
                const Tile tl = make_tile(a, &plan, it);
                const int d = i_acc & 1;
                const uint32_t shape = shape_f16(128, tl.n, !a.p.transposed);
                if (i_acc >= 2 && !bar_wait(acc_empty(d), ((i_acc >> 1) - 1) & 1, &gave_up, count))
                    break;
                fence_after();
                for (int k = k_lo; k < k_hi; k++, it_step++) {
                    const int s = it_step % kStages;
                    const uint32_t par = (it_step / kStages) & 1;
                    if (!bar_wait(full_b(s), par, &gave_up, count) || !bar_wait(full_a(s), par, &gave_up, count)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t sa = base + s * kABytes, sB = base + kStageB + s * kBBytes;
#pragma unroll
                    for (int j = 0; j < kStep / 16; j++) {
                        // 16 inputs on: 32 bytes of a row along K, two groups of 8 rows along M
                        const uint64_t da = a.p.transposed ? operand(sa + 32 * j, 16, 1024)
                                                           : operand(sa + 2048 * j, 8192, 1024);
                        mma_f16(tmem + d * kN, da, operand(sB + 32 * j, 16, 1024), shape, k > k_lo || j > 0);
                    }
                    commit(empty(s));
                }
                if (ok)
                    commit(acc_full(d));
            }
        }
    }
    __syncwarp();

    if (a.split > 1) {
        // partial sums of the cluster, added in block order
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (it0 < n_tiles && warp < kDecWarps + kOutWarps) {
            // (decode warps read what the result warps' `griddepcontrol.wait` has waited for)
            const Tile tl = make_tile(a, &plan, it0);
            const int groups = (kDecWarps + kOutWarps) * 4;
            const int mine = (tl.n + a.split - 1 - rank) / a.split;          // tokens rank, rank + split, ...
            for (int i = warp * 4; i < mine; i += groups) {
                const int row = rank + (i + (lane >> 3)) * a.split;
                const bool in = row < tl.n;
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; j++)
                    x[j] = 0.0f;
                if (in)
                    for (int b = 0; b < a.split; b++) {
                        uint32_t from;
                        asm("mapa.shared::cluster.u32 %0, %1, %2;"
                            : "=r"(from) : "r"(base + (uint32_t)row * 512u + (uint32_t)(lane & 7) * 16u), "r"(b));
#pragma unroll
                        for (int m = 0; m < 4; m++) {
                            float4 f;
                            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                         : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(from + 128u * m) : "memory");
                            x[4 * m] = __fadd_rn(x[4 * m], f.x);
                            x[4 * m + 1] = __fadd_rn(x[4 * m + 1], f.y);
                            x[4 * m + 2] = __fadd_rn(x[4 * m + 2], f.z);
                            x[4 * m + 3] = __fadd_rn(x[4 * m + 3], f.w);
                        }
                    }
                finish(a, tl, in ? tl.t0 + row : tl.hi, x, lane);
            }
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    if (gave_up) {
        // nothing may be in flight when the block ends: its last copies and matrix instructions
        if (warp == kDecWarps + kOutWarps && lane == 0)
            for (uint32_t back = 1; back <= kStages && back <= issued; back++)
                bar_drain(full_b((issued - back) % kStages), ((issued - back) / kStages) & 1);
        if (warp == kDecWarps + kOutWarps + 1 && lane == 0) {
            commit(drained);
            bar_drain(drained, 0);
        }
        __syncthreads();
    }
    if (warp == kDecWarps) {
        fence_after();
        tmem_free<512>(tmem);
    }
}

template <int K> exl3_status launch_k(const Args &a, unsigned grid, cudaStream_t s) {
    static_assert(kSmem <= 227 * 1024, "shared memory of one block");
    cudaError_t e = cudaFuncSetAttribute(product_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
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
    attr[1].val.clusterDim.x = (unsigned)a.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, product_kernel<K>, a);
    if (e != cudaSuccess)
        return cuda_check(e, "coded product launch");
    note_launch();
    return cuda_check(cudaGetLastError(), "coded product launch");
}

}  // namespace

exl3_status launch_product(const ProductLaunch &p, cudaStream_t s) {
    Args a;
    a.p = p;
    a.n_in = (int)(p.transposed ? p.cols : p.rows);
    a.n_out = (int)(p.transposed ? p.rows : p.cols);
    const int64_t sms = device_sm_count();
    // token tiles of even size, at most kN; experts' sizes are not known here
    const int64_t n = (p.T + kN - 1) / kN;
    a.tile_n = p.offsets ? kN : (int)(((p.T + n - 1) / n + 15) / 16 * 16);
    const int64_t used = p.T < p.E ? p.T : p.E;
    const int64_t tok = p.offsets ? used + (p.T + 7 * used) / kN + 1 : n;
    const int64_t tiles = tok * (a.n_out / 128);
    // blocks that would idle share the sums of the tiles, at least 4 steps each
    const int steps = a.n_in / kStep;
    a.split = 1;
    while (a.split < 8 && tiles * a.split * 2 <= sms && steps >= a.split * 2 * 4)
        a.split *= 2;
    const unsigned grid = (unsigned)(a.split > 1 ? tiles * a.split : tiles < sms ? tiles : sms);
    switch (p.K) {
    case 1: return launch_k<1>(a, grid, s);
    case 2: return launch_k<2>(a, grid, s);
    case 3: return launch_k<3>(a, grid, s);
    default: return launch_k<4>(a, grid, s);
    }
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
    *n = v;
    return EXL3_OK;
}

}  // namespace exl3
