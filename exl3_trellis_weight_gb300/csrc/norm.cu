// norm.cu -- root-mean-square norms of rows, with the residual's addition before and
// blocks in e4m3 behind them, their gradients, and the same blocks of any matrix.
//
//   h = rn(x + residual), s = 1 / sqrt(sum h^2 / n + eps), y = h s w
//   with g = dy w:  dx = s g - h s^3 sum(g h) / n (+ dh),  dw = sum over rows of dy h s
//
// All of it is bound by memory: each row is read once, stays in registers (in the 16 bits
// it came in) between its sum and its result, and the block of 128 that shares a scale lies
// in half a warp.  A warp's unit is 256 neighbouring columns: lane l has columns 8l .. 8l + 7
// of it where rows allow 16-byte accesses (kWide), pairs 2l + 64i where they are whole pairs, and
// columns l, l + 32, ... where they are not, so that a warp's accesses are whole sectors
// each way.  16384 x 4096 with a residual: 83 us, 6.4 TB/s (a copy: 6.8); one row: 5 us.  A row of
// up to 256 columns is one warp with one load of each array on its way, and below that some of its lanes
// load nothing: 131072 x 256 48 us (2.8 TB/s), 262144 x 128 85 (1.6).  8192 rows of 4096, 4098 and 4097 columns with a residual: 46, 54 and 84 us.
#include "layer.cuh"
#include "tc.cuh"

namespace exl3 {

namespace {

constexpr int kUnitN = 256;
constexpr int kSingle = 0, kWide = 1, kPairs = 2;      // VEC: a thread's accesses

// ---- eight values of a unit in the 16 bits of memory ------------------------------
struct Eight {
    uint32_t w[4];
};

template <int VEC> __device__ __forceinline__ int column(int unit, int lane, int j) {
    return unit * kUnitN + (VEC == kWide ? lane * 8 + j : VEC == kPairs ? 2 * lane + 64 * (j >> 1) + (j & 1) : lane + 32 * j);
}

template <typename T, int VEC> __device__ __forceinline__ Eight load_eight(const T *row, int unit, int lane, int n) {
    Eight e{};
    if (VEC == kWide) {
        const int c = column<kWide>(unit, lane, 0);
        if (c < n) {
            const uint4 q = *reinterpret_cast<const uint4 *>(row + c);
            e.w[0] = q.x, e.w[1] = q.y, e.w[2] = q.z, e.w[3] = q.w;
        }
    } else if (VEC == kPairs) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int c = column<VEC>(unit, lane, 2 * i);
            if (c < n)
                e.w[i] = *reinterpret_cast<const uint32_t *>(row + c);
        }
    } else {
        const uint16_t *r = reinterpret_cast<const uint16_t *>(row);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int c = column<VEC>(unit, lane, j);
            if (c < n)
                e.w[j >> 1] |= (uint32_t)r[c] << (16 * (j & 1));
        }
    }
    return e;
}

template <typename T, int VEC> __device__ __forceinline__ void store_eight(T *row, int unit, int lane, int n, const Eight &e) {
    if (VEC == kWide) {
        const int c = column<kWide>(unit, lane, 0);
        if (c < n)
            *reinterpret_cast<uint4 *>(row + c) = make_uint4(e.w[0], e.w[1], e.w[2], e.w[3]);
    } else if (VEC == kPairs) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int c = column<VEC>(unit, lane, 2 * i);
            if (c < n)
                *reinterpret_cast<uint32_t *>(row + c) = e.w[i];
        }
    } else {
        uint16_t *r = reinterpret_cast<uint16_t *>(row);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int c = column<VEC>(unit, lane, j);
            if (c < n)
                r[c] = (uint16_t)(e.w[j >> 1] >> (16 * (j & 1)));
        }
    }
}

template <typename T> __device__ __forceinline__ void unpack_eight(const Eight &e, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = unpack2<T>(e.w[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
template <typename T> __device__ __forceinline__ Eight pack_eight(const float (&v)[8]) {
    Eight e;
#pragma unroll
    for (int i = 0; i < 4; i++)
        e.w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    return e;
}

// the same from binary32, as the norm's weights may be, too
template <typename T, int VEC>
__device__ __forceinline__ void load_weights(const void *w, bool wide, int unit, int lane, int n, float (&v)[8]) {
    if (!wide) {
        unpack_eight<T>(load_eight<T, VEC>(reinterpret_cast<const T *>(w), unit, lane, n), v);
        return;
    }
    const float *f = reinterpret_cast<const float *>(w);
    if (VEC == kPairs) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int c = column<VEC>(unit, lane, 2 * i);
            const float2 q = c < n ? *reinterpret_cast<const float2 *>(f + c) : make_float2(0.0f, 0.0f);
            v[2 * i] = q.x, v[2 * i + 1] = q.y;
        }
    } else if (VEC == kWide) {
        const int c = column<kWide>(unit, lane, 0);
        float4 a = {}, b = {};
        if (c < n)
            a = reinterpret_cast<const float4 *>(f + c)[0], b = reinterpret_cast<const float4 *>(f + c)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int c = column<VEC>(unit, lane, j);
            v[j] = c < n ? f[c] : 0.0f;
        }
    }
}

// ---- blocks of 128 ------------------------------------------------------------------
// bits of the largest magnitude: as integers they order like the magnitudes, a NaN above all
__device__ __forceinline__ uint32_t top_bits(uint32_t m, float v) { return max(m, __float_as_uint(v) & 0x7FFFFFFFu); }

__device__ __forceinline__ void block_scale(uint32_t top, float &inv, float &scale) {
    const float m = __uint_as_float(max(top, kLeast8));
    inv = __fdiv_rn(kTop8, m);
    scale = __fdiv_rn(m, kTop8);
}

// A unit's eight values of each lane to codes: two blocks of 128, each half a warp (VEC)
// or half of every lane's values.  Outside of the row values are 0.
template <int VEC>
__device__ __forceinline__ void encode_row(const float (&v)[8], uint8_t *codes, float *scale, int64_t hop, int unit, int lane,
                                           int n) {
    if (VEC == kWide) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; j++)
            top = top_bits(top, v[j]);
#pragma unroll
        for (int d = 8; d; d >>= 1)
            top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        float inv, sc;
        block_scale(top, inv, sc);
        const int c = column<kWide>(unit, lane, 0);
        if (c < n) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; i++)
                q[i] = pack8(__fmul_rn(v[2 * i], inv), __fmul_rn(v[2 * i + 1], inv));
            *reinterpret_cast<uint2 *>(codes + c) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
            if ((lane & 15) == 0)
                scale[(c >> 7) * hop] = sc;
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; j++)
                top = top_bits(top, v[4 * h + j]);
            top = __reduce_max_sync(0xffffffffu, top);
            float inv, sc;
            block_scale(top, inv, sc);
#pragma unroll
            for (int j = 0; j < 4; j += VEC == kPairs ? 2 : 1) {
                const int c = column<VEC>(unit, lane, 4 * h + j);
                const uint32_t q = pack8(__fmul_rn(v[4 * h + j], inv), __fmul_rn(v[4 * h + (j + 1) % 4], inv));
                if (c < n) {
                    if (VEC == kPairs)
                        *reinterpret_cast<uint16_t *>(codes + c) = (uint16_t)q;
                    else
                        codes[c] = (uint8_t)q;
                }
            }
            const int c0 = unit * kUnitN + 128 * h;
            if (lane == 0 && c0 < n)
                scale[(c0 >> 7) * hop] = sc;
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

// A row whose sum of squares passes binary32's range (bfloat16's largest squares do) is
// summed again with its values times 2^-75: the warps of a row take that turn together.
constexpr float kDown = 0x1p-75f, kDownG = 0x1p-100f;
__device__ __forceinline__ bool passed(float sum) { return !(sum <= 0x1.fffffep127f); }
__device__ __forceinline__ void row_barrier(int sub, int wr) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(wr * 32) : "memory");
}

// ---- the norm -------------------------------------------------------------------------
// A row to `wr` warps, each VPT units of it; a block has one row or several.
template <typename T, int VEC, int VPT>
__global__ void __launch_bounds__(1024) norm_kernel(const NormLaunch a, int wr) {
    __shared__ float place[32];
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int sub = warp / wr, wi = warp % wr, rows = (int)(blockDim.x >> 5) / wr;
    const int64_t t = (int64_t)blockIdx.x * rows + sub;
    const bool in = t < a.T;
    Eight h[VPT];
    float sum = 0.0f;
    if (in) {
        const T *x = reinterpret_cast<const T *>(a.x) + t * a.x_stride;
        const T *r = reinterpret_cast<const T *>(a.residual) + t * a.r_stride;
        Eight e[VPT];
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            h[k] = load_eight<T, VEC>(x, wi + k * wr, lane, a.n);
            if (a.residual)
                e[k] = load_eight<T, VEC>(r, wi + k * wr, lane, a.n);
        }
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            float v[8];
            unpack_eight<T>(h[k], v);
            if (a.residual) {
                float u[8];
                unpack_eight<T>(e[k], u);
#pragma unroll
                for (int j = 0; j < 8; j++)
                    v[j] = __fadd_rn(v[j], u[j]);
                // what later layers read is what is normed: the rounded sum
                h[k] = pack_eight<T>(v);
                unpack_eight<T>(h[k], v);
                store_eight<T, VEC>(reinterpret_cast<T *>(a.h) + t * a.h_stride, wi + k * wr, lane, a.n, h[k]);
            }
#pragma unroll
            for (int j = 0; j < 8; j++)
                sum = __fmaf_rn(v[j], v[j], sum);
        }
    }
    sum = warp_sum(sum);
    if (wr > 1) {
        if (lane == 0)
            place[warp] = sum;
        __syncthreads();
        sum = warp_sum(lane < wr ? place[sub * wr + lane] : 0.0f);
    }
    if (!in)
        return;
    float down = 1.0f;
    if (passed(sum)) {
        down = kDown;
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            float v[8];
            unpack_eight<T>(h[k], v);
#pragma unroll
            for (int j = 0; j < 8; j++)
                sum = __fmaf_rn(__fmul_rn(v[j], kDown), __fmul_rn(v[j], kDown), sum);
        }
        sum = warp_sum(sum);
        if (wr > 1) {
            row_barrier(sub, wr);          // the first sums are read
            if (lane == 0)
                place[warp] = sum;
            row_barrier(sub, wr);
            sum = warp_sum(lane < wr ? place[sub * wr + lane] : 0.0f);
        }
    }
    const float s = __frsqrt_rn(__fmaf_rn(__fmul_rn(a.eps, down), down, __fdiv_rn(sum, (float)a.n)));
#pragma unroll
    for (int k = 0; k < VPT; k++) {
        const int unit = wi + k * wr;
        float v[8], w[8];
        unpack_eight<T>(h[k], v);
        if (down != 1.0f) {
#pragma unroll
            for (int j = 0; j < 8; j++)
                v[j] = __fmul_rn(v[j], kDown);
        }
        load_weights<T, VEC>(a.weight, a.w_dt == EXL3_F32, unit, lane, a.n, w);
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[j] = __fmul_rn(__fmul_rn(v[j], s), w[j]);
        if (a.y)
            store_eight<T, VEC>(reinterpret_cast<T *>(a.y) + t * a.y_stride, unit, lane, a.n, pack_eight<T>(v));
        if (a.y8) {
            if (VEC == kWide ? column<kWide>(unit, lane, 0) >= a.n : false) {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    v[j] = 0.0f;
            } else if (VEC != kWide) {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    v[j] = column<VEC>(unit, lane, j) < a.n ? v[j] : 0.0f;
            }
            encode_row<VEC>(v, a.y8 + t * a.n, a.scale + t, a.T, unit, lane, a.n);
        }
    }
}

// Binary32 in pairs, each half rounded as the single operation would be: half the instructions,
// which with 20 to a value bound the gradients as much as memory does.
struct Pair {
    float x, y;
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\t"
        "mov.b64 {%0, %1}, c;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
template <typename T> __device__ __forceinline__ void unpack_pairs(const Eight &e, Pair (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = unpack2<T>(e.w[i]);
        v[i] = {f.x, f.y};
    }
}

// ---- its gradients ----------------------------------------------------------------------
// Blocks stay and take rows in turn, the next rows on their way while one is summed: a thread
// keeps its columns' part of dweight, in registers up to two units and in shared memory
// beyond, where registers run out.
// RING: whole rows are copied into stages of shared memory, `depth` of them ahead.  (One row
// ahead in registers were 48 KB to an SM on their way: 8192 x 4096 took 66 us, 4.1 TB/s; now
// 52, 5.2 TB/s, and 5 for the sum of dweight's parts, whose launch overlaps.  In what is left a
// row's wait for its copy, its sums, the meeting of its warps and its results follow one another,
// with 16 warps to an SM to fill the gaps.)
// WAY: the next row is asked for into registers.
__device__ unsigned int g_norm_timeouts;
constexpr int kMaxDepth = 8;

template <typename T, int VEC, int VPT, bool WAY, bool RING>
__global__ void __launch_bounds__(RING ? 512 : 1024, RING && VPT == 1 ? 2 : 1) norm_grad_kernel(const NormGradLaunch a, int wr, int depth) {
    constexpr bool kRegs = VPT <= 2;
    __shared__ float2 place[2][32];
    __shared__ __align__(8) unsigned long long bars[RING ? kMaxDepth : 1];
    __shared__ int gave_up;
    extern __shared__ __align__(16) float dw_mem[];
    // (the sum of dweight's parts waits for this kernel's end)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int sub = warp / wr, wi = warp % wr, rows = (int)(blockDim.x >> 5) / wr;
    const bool want = a.dweight != nullptr, wide = a.w_dt == EXL3_F32;
    Pair dw[kRegs ? VPT : 1][4];
    const float inv_n = __fdiv_rn(1.0f, (float)a.n);
    float *const mine = dw_mem + threadIdx.x;            // [unit][value][thread]
    if (kRegs) {
#pragma unroll
        for (int k = 0; k < (kRegs ? VPT : 1); k++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                dw[k][j] = {0.0f, 0.0f};
    } else if (want) {
        for (int k = 0; k < VPT * 8; k++)
            mine[k * blockDim.x] = 0.0f;
    }
    const T *const dy = reinterpret_cast<const T *>(a.dy), *const hs = reinterpret_cast<const T *>(a.h);
    const T *const ds = reinterpret_cast<const T *>(a.dh);
    const int64_t step = (int64_t)gridDim.x * rows;
    Eight eg[VPT], eh[VPT], ed[VPT];
    auto fetch = [&](int64_t t, Eight (&g)[VPT], Eight (&h)[VPT], Eight (&d)[VPT]) {
#pragma unroll
        for (int k = 0; k < VPT; k++) {
            g[k] = h[k] = d[k] = Eight{};
            if (t < a.T) {
                g[k] = load_eight<T, VEC>(dy + t * a.dy_stride, wi + k * wr, lane, a.n);
                h[k] = load_eight<T, VEC>(hs + t * a.h_stride, wi + k * wr, lane, a.n);
                if (ds)
                    d[k] = load_eight<T, VEC>(ds + t * a.dh_stride, wi + k * wr, lane, a.n);
            }
        }
    };
    if (WAY)
        fetch((int64_t)blockIdx.x * rows + sub, eg, eh, ed);
    // stage: dy, h and dh of the block's rows, one behind the other
    const uint32_t ring = tc::saddr(dw_mem), bar0 = tc::saddr(bars), row_bytes = (uint32_t)a.n * 2u;
    const int ops = ds ? 3 : 2;
    const uint32_t stage_bytes = (uint32_t)(ops * rows) * row_bytes;
    auto issue = [&](int64_t t0, int s) {  // by a warp
        if (t0 >= a.T)
            return;
        const int n = (int)min((int64_t)rows, a.T - t0);
        if (lane == 0)
            tc::bar_expect(bar0 + 8u * s, (uint32_t)(ops * n) * row_bytes);
        __syncwarp();
        const int op = lane / rows, r = lane % rows;
        if (op < ops && r < n) {
            const T *from = op == 0 ? dy + (t0 + r) * a.dy_stride : op == 1 ? hs + (t0 + r) * a.h_stride : ds + (t0 + r) * a.dh_stride;
            tc::bulk_load(ring + s * stage_bytes + (uint32_t)(op * rows + r) * row_bytes, from, row_bytes, bar0 + 8u * s);
        }
        __syncwarp();
    };
    if constexpr (RING) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < depth; s++)
                tc::bar_init(bar0 + 8u * s, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            gave_up = 0;
        }
        __syncthreads();
        if (warp == 0)
            for (int s = 0; s < depth; s++)
                issue((int64_t)(blockIdx.x + (int64_t)s * gridDim.x) * rows, s);
    }
    int stage = 0;
    uint32_t phase = 0;
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.T; t0 += step, turn ^= 1) {
        const int64_t t = t0 + sub;
        const bool in = t < a.T;
        float eps = a.eps;
        Eight ng[WAY ? VPT : 1], nh[WAY ? VPT : 1], nd[WAY ? VPT : 1];
        if constexpr (RING) {
            tc::bar_wait(bar0 + 8u * stage, phase, &gave_up, &g_norm_timeouts);
            const char *at = reinterpret_cast<const char *>(dw_mem) + stage * stage_bytes + sub * row_bytes;
#pragma unroll
            for (int k = 0; k < VPT; k++) {
                const int c = column<kWide>(wi + k * wr, lane, 0);
                auto take = [&](int op) {
                    Eight e{};
                    if (in && c < a.n) {
                        const uint4 q = *reinterpret_cast<const uint4 *>(at + (size_t)op * rows * row_bytes + 2 * c);
                        e.w[0] = q.x, e.w[1] = q.y, e.w[2] = q.z, e.w[3] = q.w;
                    }
                    return e;
                };
                eg[k] = take(0);
                eh[k] = take(1);
                if (ds)
                    ed[k] = take(2);
            }
        } else if constexpr (WAY) {
            fetch(t + step, ng, nh, nd);
        } else {
            fetch(t, eg, eh, ed);
        }
        // dy, h and dy weight of a unit: they stay in registers where there are some, and are
        // unpacked again for the results where there are not
        constexpr bool kStay = VPT == 1 || RING;
        struct Unit {
            Pair g[4], v[4], gw[4];
        } stay[kStay ? VPT : 1];
        float hh, gh, dh = 1.0f, dg = 1.0f;                  // (powers of two, see below)
        auto unit = [&](int k, Unit &u) {
            unpack_pairs<T>(eg[k], u.g);
            unpack_pairs<T>(eh[k], u.v);
            float w[8];
            load_weights<T, VEC>(a.weight, wide, wi + k * wr, lane, a.n, w);
#pragma unroll
            for (int j = 0; j < 4; j++)
                u.gw[j] = mul2(u.g[j], {w[2 * j], w[2 * j + 1]});
        };
        auto down = [&](Unit &u, float fh, float fg) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                u.v[j] = mul2(u.v[j], {fh, fh});
                u.gw[j] = mul2(u.gw[j], {fg, fg});
            }
        };
        // (of h times fh and dy weight times fg, beside what they have been multiplied by before)
        auto sums = [&](bool first, float fh, float fg) {
            Pair h2 = {0.0f, 0.0f}, g2 = {0.0f, 0.0f};
            dh = __fmul_rn(dh, fh);
            dg = __fmul_rn(dg, fg);
#pragma unroll
            for (int k = 0; k < VPT; k++) {
                Unit &u = stay[kStay ? k : 0];
                if (first || !kStay)
                    unit(k, u);
                if (!first)
                    down(u, kStay ? fh : dh, kStay ? fg : dg);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    h2 = fma2(u.v[j], u.v[j], h2);
                    g2 = fma2(u.gw[j], u.v[j], g2);
                }
            }
            hh = warp_sum(__fadd_rn(h2.x, h2.y));
            gh = warp_sum(__fadd_rn(g2.x, g2.y));
        };
        sums(true, 1.0f, 1.0f);
        if (wr > 1) {
            // (two places in turn: a row's reads are done before the barrier of the next)
            if (lane == 0)
                place[turn][warp] = make_float2(hh, gh);
            __syncthreads();
            if (RING) {                    // (everyone has read the stage)
                if (warp == 0)
                    issue(t0 + depth * step, stage);
                if (++stage == depth)
                    stage = 0, phase ^= 1;
            }
            const float2 q = lane < wr ? place[turn][sub * wr + lane] : make_float2(0.0f, 0.0f);
            hh = warp_sum(q.x);
            gh = warp_sum(q.y);
        }
        if (in) {
            // beyond binary32's range: h, and then dy weight if that was not enough, times powers of
            // two (each at once as well, the products of small dy with large h were lost below)
            float back = 1.0f;
            if (passed(hh) || passed(fabsf(gh))) {
#pragma unroll 1
                for (int again = 0; again < 2; again++) {
                    const bool of_h = dh == 1.0f && passed(hh), of_g = dg == 1.0f && passed(fabsf(gh));
                    if (!of_h && !of_g)
                        break;
                    sums(false, of_h ? kDown : 1.0f, of_h ? 1.0f : kDownG);
                    if (wr > 1) {
                        row_barrier(sub, wr);  // the sums before are read
                        if (lane == 0)
                            place[turn][warp] = make_float2(hh, gh);
                        row_barrier(sub, wr);
                        const float2 q = lane < wr ? place[turn][sub * wr + lane] : make_float2(0.0f, 0.0f);
                        hh = warp_sum(q.x);
                        gh = warp_sum(q.y);
                    }
                }
                back = __fdiv_rn(dh, dg);
                eps = __fmul_rn(__fmul_rn(a.eps, dh), dh);
            }
            // with h' = h dh, g' = dy weight dg, s' = s / dh:  dx = s' dh / dg (g' - h' s'^2 sum(g' h') / n)
            const float s = __frsqrt_rn(__fmaf_rn(hh, inv_n, eps));
            const float c = -__fmul_rn(__fmul_rn(s, s), __fmul_rn(gh, inv_n)), sd = __fmul_rn(s, back);
#pragma unroll
            for (int k = 0; k < VPT; k++) {
                Unit &u = stay[kStay ? k : 0];
                if (!kStay) {
                    unit(k, u);
                    if (dh != 1.0f || dg != 1.0f)
                        down(u, dh, dg);
                }
                if (want) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const Pair p = mul2(u.v[j], {s, s});
                        if (kRegs) {
                            Pair &d = dw[kRegs ? k : 0][j];
                            d = fma2(u.g[j], p, d);
                        } else {
                            float *d = mine + (k * 8 + 2 * j) * blockDim.x;
                            d[0] = __fmaf_rn(u.g[j].x, p.x, d[0]);
                            d[blockDim.x] = __fmaf_rn(u.g[j].y, p.y, d[blockDim.x]);
                        }
                    }
                }
                Eight e;
                Pair o[4];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    o[j] = mul2(fma2(u.v[j], {c, c}, u.gw[j]), {sd, sd});
                if (ds) {
                    unpack_pairs<T>(ed[k], u.g);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        o[j] = add2(o[j], u.g[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; j++)
                    e.w[j] = pack2<T>(o[j].x, o[j].y);
                store_eight<T, VEC>(reinterpret_cast<T *>(a.dx) + t * a.dx_stride, wi + k * wr, lane, a.n, e);
            }
        }
        if constexpr (WAY) {
#pragma unroll
            for (int k = 0; k < VPT; k++)
                eg[k] = ng[k], eh[k] = nh[k], ed[k] = nd[k];
        }
    }
    if (RING && gave_up && threadIdx.x == 0)           // nothing may be in flight when the block ends
        for (int s = 0; s < depth; s++)
            tc::bar_drain(bar0 + 8u * s, phase ^ (s < stage));
    if (!want)
        return;
    float *part = a.part + ((int64_t)blockIdx.x * rows + sub) * a.n;
#pragma unroll
    for (int k = 0; k < VPT; k++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int c = column<VEC>(wi + k * wr, lane, j);
            if (c < a.n)
                part[c] = !kRegs ? mine[(k * 8 + j) * blockDim.x] : j & 1 ? dw[kRegs ? k : 0][j >> 1].y : dw[kRegs ? k : 0][j >> 1].x;
        }
}

// dweight: the partial rows of 32 columns, 32 threads to a column, in a fixed order
template <typename T> __global__ void __launch_bounds__(1024) dweight_kernel(const float *part, int parts, int n, void *out, bool wide) {
    __shared__ float place[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c < n) {
#pragma unroll 8
        for (int i = warp; i < parts; i += 32)
            s = __fadd_rn(s, __ldcg(part + (int64_t)i * n + c));
    }
    place[warp][lane] = s;
    __syncthreads();
    s = warp_sum(place[lane][warp]);
    const int d = blockIdx.x * 32 + warp;
    if (lane == 0 && d < n) {
        if (wide)
            reinterpret_cast<float *>(out)[d] = s;
        else
            reinterpret_cast<T *>(out)[d] = from_f32<T>(s);
    }
}

// ---- blocks of any matrix ---------------------------------------------------------------
template <typename T, int VEC> __device__ __forceinline__ void load_values(const T *row, int unit, int lane, int n, float (&v)[8]) {
    if constexpr (sizeof(T) == 4)
        load_weights<__half, VEC>(row, true, unit, lane, n, v);
    else
        unpack_eight<T>(load_eight<T, VEC>(row, unit, lane, n), v);
}

// 1 x 128: a warp takes four units, one behind the other.  1001 x 12288: 10 us, of which 4 are any
// kernel's ends and 5.5 the bytes at a copy's rate; it runs in two and a half rounds of blocks, whose
// 63 registers a thread (values in binary32) leave room for four to an SM.  Replayed graphs with 1, 2,
// 4 and 8 units a warp: 8192 x 4096 26.7, 26.2, 24.7 and 30.2 us; 1001 x 12288 13.4, 13.1, 13.2 and 16.5;
// 333 x 2000 4.1, 4.6, 5.1 and 6.2.
constexpr int kUnitsWarp = 4;
template <typename T, int VEC> __global__ void __launch_bounds__(256) rows8_kernel(const Quantize8Launch a) {
    // (a product behind this launch may load its weights; it waits for this kernel's end
    // before it reads what is written here)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, n = (int)a.n;
    const int units = (n + kUnitN - 1) / kUnitN;
    const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kUnitsWarp;
    int64_t t[kUnitsWarp];
    int unit[kUnitsWarp];
    t[0] = first / units;
    unit[0] = (int)(first - t[0] * units);
#pragma unroll
    for (int k = 1; k < kUnitsWarp; k++) {
        const bool end = unit[k - 1] + 1 == units;
        t[k] = t[k - 1] + end;
        unit[k] = end ? 0 : unit[k - 1] + 1;
    }
    float v[kUnitsWarp][8];
#pragma unroll
    for (int k = 0; k < kUnitsWarp; k++)
        load_values<T, VEC>(reinterpret_cast<const T *>(a.x) + t[k] * a.stride, unit[k], lane, t[k] < a.T ? n : 0, v[k]);
#pragma unroll
    for (int k = 0; k < kUnitsWarp; k++)
        encode_row<VEC>(v[k], a.codes + t[k] * n, a.scale + t[k], a.T, unit[k], lane, t[k] < a.T ? n : 0);
}

// 128 x 128: eight warps to a block, two rows of it a warp at a time.  12288 x 4096 from bfloat16: 27 us,
// 5.6 TB/s.
template <typename T, int VEC> __global__ void __launch_bounds__(256) blocks8_kernel(const Quantize8Launch a) {
    __shared__ uint32_t place[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks_c = (int)((a.n + 127) / 128);
    const int64_t r0 = (int64_t)(blockIdx.x / blocks_c) * 128;
    const int c0 = (int)(blockIdx.x % blocks_c) * 128, cols = (int)min((int64_t)128, a.n - c0);
    // (a unit of 256 values: rows 2i, 2i + 1 of the block.  They stay in the form they came in:
    // as 64 numbers of binary32 they left room for three blocks an SM)
    constexpr int kWords = sizeof(T) == 4 ? 8 : 4;
    uint32_t raw[8][kWords];
    auto values = [&](int i, float (&v)[8]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 8; j++)
                v[j] = __uint_as_float(raw[i][j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 f = unpack2<T>(raw[i][j]);
                v[2 * j] = f.x, v[2 * j + 1] = f.y;
            }
        }
    };
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t r = r0 + 2 * (warp + 8 * i) + (VEC ? lane >> 4 : 0);
        const T *row = reinterpret_cast<const T *>(a.x) + r * a.stride + c0;
        if constexpr (VEC) {
            const int c = (lane & 15) * 8;
            const bool in = r < a.T && c < cols;
#pragma unroll
            for (int j = 0; j < kWords; j += 4) {
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
                if (in)
                    q = *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(row + c) + 4 * j);
                raw[i][j] = q.x, raw[i][j + 1] = q.y, raw[i][j + 2] = q.z, raw[i][j + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int c = lane + 32 * (j & 3);
                const bool in = r + (j >> 2) < a.T && c < cols;
                const T *at = row + (j >> 2) * a.stride + c;
                if constexpr (sizeof(T) == 4) {
                    raw[i][j] = in ? *reinterpret_cast<const uint32_t *>(at) : 0u;
                } else {
                    const uint32_t w = in ? *reinterpret_cast<const uint16_t *>(at) : 0u;
                    raw[i][j >> 1] = j & 1 ? raw[i][j >> 1] | w << 16 : w;
                }
            }
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float v[8];
        values(i, v);
#pragma unroll
        for (int j = 0; j < 8; j++)
            top = top_bits(top, v[j]);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0)
        place[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, place[lane & 7]);
    float inv, sc;
    block_scale(top, inv, sc);
    if (threadIdx.x == 0)
        a.scale[blockIdx.x] = sc;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float v[8];
        values(i, v);
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            q[j] = pack8(__fmul_rn(v[2 * j], inv), __fmul_rn(v[2 * j + 1], inv));
        if (VEC) {
            const int64_t r = r0 + 2 * (warp + 8 * i) + (lane >> 4);
            const int c = (lane & 15) * 8;
            if (r < a.T && c < cols)
                *reinterpret_cast<uint2 *>(a.codes + r * a.n + c0 + c) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int64_t r = r0 + 2 * (warp + 8 * i) + (j >> 2);
                const int c = lane + 32 * (j & 3);
                if (r < a.T && c < cols)
                    a.codes[r * a.n + c0 + c] = (uint8_t)(q[j >> 1] >> (8 * (j & 1)));
            }
        }
    }
}

// ---- launches -----------------------------------------------------------------------------
// rows whose elements, 8 or 2 at a time (see column), all stand at multiples of their size; the
// narrowest of several arrays counts
int access_of(const void *p, int64_t stride, int size, int64_t n, int best) {
    if (!p)
        return best;
    auto fits = [&](int bytes) { return (uintptr_t)p % bytes == 0 && stride * size % bytes == 0; };
    const int own = n % 8 == 0 && fits(size == 1 ? 8 : 16) ? kWide : n % 2 == 0 && fits(2 * size) ? kPairs : kSingle;
    return own == kWide ? best : best == kWide || own == kSingle ? own : best;
}

struct Shape {
    int vpt, wr, rows;        // units of a warp, warps of a row, rows of a block
};

// As many units a warp, up to four, as leave 16 warps to an SM: its loads are longer and a row
// meets in fewer warps.  (16384 x 4096 with four, two and one units a warp: 83, 90 and
// 104 us; 16384 x 1024 with four and one: 27 and 39; 333 x 4096 with four and two: 7.2 and 6.2.)
Shape norm_shape(int64_t T, int64_t n) {
    const int units = (int)((n + kUnitN - 1) / kUnitN);
    const int64_t sms = device_sm_count();
    Shape f;
    f.vpt = 1;
    while (f.vpt < 4 && (units > 32 * f.vpt || (units > f.vpt && T * ((units + 2 * f.vpt - 1) / (2 * f.vpt)) >= 16 * sms)))
        f.vpt *= 2;
    f.wr = (units + f.vpt - 1) / f.vpt;
    f.rows = T > 2 * sms && f.wr < 8 ? 8 / f.wr : 1;
    return f;
}

template <typename T, int VEC> exl3_status norm_v(const NormLaunch &p, const Shape &f, cudaStream_t s) {
    const unsigned grid = (unsigned)((p.T + f.rows - 1) / f.rows), block = (unsigned)(f.rows * f.wr * 32);
    if (f.vpt == 1)
        norm_kernel<T, VEC, 1><<<grid, block, 0, s>>>(p, f.wr);
    else if (f.vpt == 2)
        norm_kernel<T, VEC, 2><<<grid, block, 0, s>>>(p, f.wr);
    else
        norm_kernel<T, VEC, 4><<<grid, block, 0, s>>>(p, f.wr);
    note_launch();
    return cuda_check(cudaGetLastError(), "norm launch");
}

template <typename T> exl3_status norm_t(const NormLaunch &p, int vec, const Shape &f, cudaStream_t s) {
    return vec == kWide ? norm_v<T, kWide>(p, f, s) : vec == kPairs ? norm_v<T, kPairs>(p, f, s) : norm_v<T, kSingle>(p, f, s);
}

// Warps of an SM (half of them with two units each, which take 117 registers), and how many
// columns a ring of whole rows is for.  (8192 rows, with and without: 512 columns 24.0 and 26.6 us,
// 1024 29 and 30, 2048 39 and 43, 8192 102 and 144.  A row of one warp has no meeting at which
// its stage could be asked for again.)
constexpr int kGradWarps = 32, kRingFrom = 512, kRingTo = 8192;
static_assert(kRingFrom > kUnitN, "two warps to a row at least");
constexpr uint32_t kRingRoom = 208 * 1024;     // of an SM

struct GradShape : Shape {
    int depth;                // 0: no ring
    int per_sm;               // blocks
};
GradShape grad_shape(int64_t n, bool ring, bool with_dh) {
    const int units = (int)((n + kUnitN - 1) / kUnitN);
    GradShape f;
    // (ring, 16384 x 4096: two units a warp 98 us, one 110; 1000 x 1024: 16.4 and 14.7)
    f.vpt = ring ? (units <= 8 ? 1 : 2) : units <= 16 ? 1 : units <= 64 ? 2 : 4;
    f.wr = (units + f.vpt - 1) / f.vpt;
    f.rows = f.wr < 8 ? 8 / f.wr : 1;
    f.per_sm = (ring && f.vpt == 2 ? kGradWarps / 2 : kGradWarps) / (f.rows * f.wr);
    f.per_sm = f.per_sm > 0 ? f.per_sm : 1;
    f.depth = 0;
    if (ring) {
        const uint32_t stage = (uint32_t)((with_dh ? 3 : 2) * f.rows * n * 2);
        f.depth = (int)(kRingRoom / (f.per_sm * stage));
        f.depth = f.depth > kMaxDepth ? kMaxDepth : f.depth;
    }
    return f;
}
unsigned grad_grid(int64_t T, const GradShape &f) {
    const int64_t most = device_sm_count() * (int64_t)f.per_sm, want = (T + f.rows - 1) / f.rows;
    return (unsigned)(want < most ? want : most);
}
bool ring_size(int64_t n) { return n >= kRingFrom && n <= kRingTo && n % 8 == 0; }

template <typename T, int VEC, int VPT, bool RING> exl3_status norm_grad_k(const NormGradLaunch &p, const GradShape &f, cudaStream_t s) {
    const unsigned block = (unsigned)(f.rows * f.wr * 32), grid = grad_grid(p.T, f);
    const size_t smem = RING ? (size_t)f.depth * (p.dh ? 3 : 2) * f.rows * p.n * 2
                             : VPT > 2 && p.dweight ? (size_t)VPT * 8 * block * sizeof(float) : 0;
    constexpr bool kWay = !RING && VPT == 1;
    if (smem) {
        const cudaError_t e = allow_smem((const void *)norm_grad_kernel<T, VEC, VPT, kWay, RING>, smem);
        if (e != cudaSuccess)
            return cuda_check(e, "cudaFuncSetAttribute(norm gradient)");
    }
    norm_grad_kernel<T, VEC, VPT, kWay, RING><<<grid, block, smem, s>>>(p, f.wr, f.depth);
    note_launch();
    return cuda_check(cudaGetLastError(), "norm gradient launch");
}
template <typename T, int VEC> exl3_status norm_grad_v(const NormGradLaunch &p, const GradShape &f, cudaStream_t s) {
    return f.vpt == 1   ? norm_grad_k<T, VEC, 1, false>(p, f, s)
           : f.vpt == 2 ? norm_grad_k<T, VEC, 2, false>(p, f, s)
                        : norm_grad_k<T, VEC, 4, false>(p, f, s);
}
template <typename T> exl3_status norm_grad_t(const NormGradLaunch &p, int vec, cudaStream_t s) {
    const GradShape r = grad_shape(p.n, vec == kWide && ring_size(p.n), p.dh != nullptr);
    const GradShape f = r.depth >= 2 ? r : grad_shape(p.n, false, false);
    if (p.T) {
        exl3_status st;
        if (f.depth)
            st = f.vpt == 1 ? norm_grad_k<T, kWide, 1, true>(p, f, s) : norm_grad_k<T, kWide, 2, true>(p, f, s);
        else
            st = vec == kWide    ? norm_grad_v<T, kWide>(p, f, s)
                 : vec == kPairs ? norm_grad_v<T, kPairs>(p, f, s)
                                 : norm_grad_v<T, kSingle>(p, f, s);
        if (st != EXL3_OK)
            return st;
    }
    if (!p.dweight)
        return EXL3_OK;
    const int parts = p.T ? (int)grad_grid(p.T, f) * f.rows : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.n + 31) / 32));
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.T ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, dweight_kernel<T>, (const float *)p.part, parts, p.n, p.dweight, p.w_dt == EXL3_F32);
    if (e != cudaSuccess)
        return cuda_check(e, "norm weight gradient launch");
    note_launch();
    return cuda_check(cudaGetLastError(), "norm weight gradient launch");
}

template <typename T> exl3_status quantize8_t(const Quantize8Launch &p, cudaStream_t s) {
    const int vec = access_of(p.codes, p.n, 1, p.n, access_of(p.x, p.stride, sizeof(T), p.n, kWide));
    if (p.block_rows == 1) {
        const int64_t units = p.T * ((p.n + kUnitN - 1) / kUnitN);
        const unsigned grid = (unsigned)((units + 8 * kUnitsWarp - 1) / (8 * kUnitsWarp));
        if (vec == kWide)
            rows8_kernel<T, kWide><<<grid, 256, 0, s>>>(p);
        else if (vec == kPairs)
            rows8_kernel<T, kPairs><<<grid, 256, 0, s>>>(p);
        else
            rows8_kernel<T, kSingle><<<grid, 256, 0, s>>>(p);
    } else {
        const unsigned grid = (unsigned)((p.n + 127) / 128 * ((p.T + 127) / 128));
        if (vec == kWide)
            blocks8_kernel<T, kWide><<<grid, 256, 0, s>>>(p);
        else
            blocks8_kernel<T, kSingle><<<grid, 256, 0, s>>>(p);
    }
    note_launch();
    return cuda_check(cudaGetLastError(), "8-bit blocks launch");
}

}  // namespace

exl3_status launch_norm(const NormLaunch &p, cudaStream_t s) {
    if (p.T == 0)
        return EXL3_OK;
    int vec = access_of(p.weight, p.n, p.w_dt == EXL3_F32 ? 4 : 2, p.n, access_of(p.x, p.x_stride, 2, p.n, kWide));
    if (p.residual)
        vec = access_of(p.h, p.h_stride, 2, p.n, access_of(p.residual, p.r_stride, 2, p.n, vec));
    vec = access_of(p.y8, p.n, 1, p.n, access_of(p.y, p.y_stride, 2, p.n, vec));
    const Shape f = norm_shape(p.T, p.n);
    return p.dt == EXL3_BF16 ? norm_t<__nv_bfloat16>(p, vec, f, s) : norm_t<__half>(p, vec, f, s);
}

int64_t norm_grad_parts(int64_t T, int64_t n) {
    if (T == 0)
        return 0;
    // (which form it is goes by alignment, too)
    const GradShape f = grad_shape(n, false, false), r = grad_shape(n, ring_size(n), false);
    const int64_t a = (int64_t)grad_grid(T, f) * f.rows, b = (int64_t)grad_grid(T, r) * r.rows;
    return a > b ? a : b;
}

exl3_status norm_take_wait_timeouts(unsigned int *n) {
    *n = 0;
    unsigned int v = 0;
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_norm_timeouts, sizeof v);
    if (e == cudaSuccess && v != 0)
        e = cudaMemcpyToSymbol(g_norm_timeouts, &zero, sizeof zero);
    if (e != cudaSuccess)
        return cuda_check(e, "wait timeout count");
    *n = v;
    return EXL3_OK;
}

exl3_status launch_norm_grad(const NormGradLaunch &p, cudaStream_t s) {
    int vec = access_of(p.dy, p.dy_stride, 2, p.n, access_of(p.h, p.h_stride, 2, p.n, kWide));
    vec = access_of(p.weight, p.n, p.w_dt == EXL3_F32 ? 4 : 2, p.n, vec);
    vec = access_of(p.dh, p.dh_stride, 2, p.n, access_of(p.dx, p.dx_stride, 2, p.n, vec));
    return p.dt == EXL3_BF16 ? norm_grad_t<__nv_bfloat16>(p, vec, s) : norm_grad_t<__half>(p, vec, s);
}

exl3_status launch_quantize8(const Quantize8Launch &p, cudaStream_t s) {
    if (p.T == 0)
        return EXL3_OK;
    return p.dt == EXL3_F32 ? quantize8_t<float>(p, s) : p.dt == EXL3_BF16 ? quantize8_t<__nv_bfloat16>(p, s) : quantize8_t<__half>(p, s);
}

}  // namespace exl3
