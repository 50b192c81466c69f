// linear_few.cuh -- what the kernels for few tokens share (linear_few.cu, expert_up.cu,
// expert_down.cu): 16 x 16 tiles of codes as the A fragments of m16n8k16 instructions.
#pragma once

#include "linear_decode.cuh"
#include "tc.cuh"

namespace exl3 {

constexpr int kTilesAhead = 16;            // tiles in a warp's ring

// PrepLaunch::order that lane_of wants: lane j's four inputs are places 4j .. 4j + 3 of 16
inline int few_order(int K, bool transposed) { return !transposed || K == 3 ? 0 : K == 1 ? 2 : 1; }

__device__ __forceinline__ uint32_t lds(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
// 16 bits of t, `B` bits before its end
template <int B> __device__ __forceinline__ uint32_t cut(uint32_t t) {
    if constexpr (B % 8 == 0)
        return __byte_perm(t, 0u, B == 0 ? 0x4410 : B == 8 ? 0x4421 : 0x4432);
    else
        return (t >> B) & 0xFFFFu;
}

// Where a lane's windows lie in a tile, in words; the same for all tiles.
// Which four inputs of 16 lane j takes follows from the codes: windows whose
// distance is a whole number of bytes come out of one shifted word in one
// instruction each (x W^^T; in x W^ a lane takes rows 4j .. 4j + 3, and outputs
// g and g + 8 where eight weights are one or two bytes).  The activations are
// stored in that order (few_order).
struct Lane {
    uint32_t last, before, sh;             // byte offsets of the first row's word and of the one before it
    uint32_t last1, sh1;                   // x W^ at K = 3: of the second row
};

template <int K, bool TR> __device__ __forceinline__ Lane lane_of(int g, int j) {
    Lane l;
    auto at = [&](int end, uint32_t &last, uint32_t &before, uint32_t &sh) {
        const int w = (end - 1) >> 5;
        last = 4u * w;
        before = 4u * (w == 0 ? 8 * K - 1 : w - 1);        // the stream is a ring
        sh = (32u - (end & 31)) & 31u;
    };
    uint32_t unused;
    if constexpr (TR)
        at(K == 1 ? 16 * g + 2 * j + 10 : K == 2 ? 32 * g + 2 * j + 26 : K == 3 ? 48 * g + 12 * j + 12 : 64 * g + 4 * j + 20,
           l.last, l.before, l.sh);
    else
        at(K <= 2 ? (64 * j + g + 9) * K : (64 * j + 2 * g + 2) * K, l.last, l.before, l.sh);
    l.last1 = l.sh1 = 0;
    if constexpr (!TR && K == 3)
        at((64 * j + 16 + 2 * g + 2) * K, l.last1, unused, l.sh1);
    return l;
}

// A fragment of one tile; `tile` is its codes' shared-memory address
template <int K, bool TR> __device__ __forceinline__ void fragment(uint32_t tile, const Lane &l, uint32_t (&a)[4]) {
    if constexpr (TR) {
        // rows g and g + 8 (4 K words on, where no word is the ring's first)
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t at = tile + l.last + 16 * K * h;
            const uint32_t w1 = lds(at), w0 = h ? lds(at - 4) : lds(tile + l.before);
            const uint32_t t = __funnelshift_r(w1, w0, l.sh);
            if constexpr (K == 1) {        // inputs 2j, 2j + 1, 2j + 8, 2j + 9
                const uint32_t u = t >> 1;
                a[h] = levels2(cut<8>(u), cut<8>(t));
                a[2 + h] = levels2(cut<0>(u), cut<0>(t));
            } else if constexpr (K == 2) { // inputs j, j + 4, j + 8, j + 12
                const uint32_t u = __funnelshift_r(w1, w0, l.sh + 24);
                a[h] = levels2(cut<0>(u), cut<16>(t));
                a[2 + h] = levels2(cut<8>(t), cut<0>(t));
            } else if constexpr (K == 3) { // inputs 4j .. 4j + 3
                a[h] = levels2(cut<9>(t), cut<6>(t));
                a[2 + h] = levels2(cut<3>(t), cut<0>(t));
            } else {                       // inputs j, j + 4; j + 8, j + 12 end a word later
                const uint32_t u = __funnelshift_r(lds(at + 4), w1, l.sh);
                a[h] = levels2(cut<16>(t), cut<0>(t));
                a[2 + h] = levels2(cut<16>(u), cut<0>(u));
            }
        }
    } else {
        // rows 4j .. 4j + 3; two outputs of each
        uint32_t w[4][2];
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const bool odd3 = K == 3 && (r & 1);
            const uint32_t at = tile + (odd3 ? l.last1 : l.last) + 4 * (K == 1 ? r >> 1 : K == 3 ? 3 * (r >> 1) : r * K / 2);
            const bool first = r == 0 || (K == 1 && r == 1);
            const uint32_t sh = K == 1 ? l.sh - 16 * (r & 1) : odd3 ? l.sh1 : l.sh;
            const uint32_t t = __funnelshift_r(lds(at), first ? lds(tile + l.before) : lds(at - 4), sh);
            w[r][0] = cut<K == 1 ? 8 : K == 2 ? 16 : K>(t);
            w[r][1] = cut<0>(t);
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            a[h] = levels2(w[0][h], w[1][h]);
            a[2 + h] = levels2(w[2][h], w[3][h]);
        }
    }
}

__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace exl3
