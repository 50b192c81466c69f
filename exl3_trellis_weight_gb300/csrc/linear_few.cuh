// linear_few.cuh -- what the kernels for few tokens share (linear_few.cu, expert_up.cu,
// expert_down.cu): 16 x 16 tiles of codes as the A fragments of m16n8k16 instructions.
#pragma once

#include "linear_decode.cuh"
#include "tc.cuh"

namespace exl3 {

constexpr int kTilesAhead = 16;            // tiles in a warp's ring

// a word of shared memory, OFF bytes behind `at`
template <int OFF> __device__ __forceinline__ uint32_t lds(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(v) : "r"(at), "n"(OFF));
    return v;
}
// two neighbouring words of shared memory, OFF bytes behind `at`
template <int OFF> __device__ __forceinline__ void lds2(uint32_t at, uint32_t &b0, uint32_t &b1) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2 + %3];" : "=r"(b0), "=r"(b1) : "r"(at), "n"(OFF));
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

// Where a lane's words lie in a warp's ring: the same distance from tile to tile, so that
// the tiles of a group are told apart in the instructions (an address of its own for each
// word made a tile 85 instructions instead of 70).
struct Words {
    uint32_t last, before, last1;
    __device__ __forceinline__ Words(uint32_t tiles, const Lane &l) : last(tiles + l.last), before(tiles + l.before), last1(tiles + l.last1) {}
    __device__ __forceinline__ void move(uint32_t by) { last += by, before += by, last1 += by; }
};

// A fragment of the tile OFF bytes on
template <int K, bool TR, int OFF> __device__ __forceinline__ void fragment(const Words &at, const Lane &l, uint32_t (&a)[4]) {
    if constexpr (TR) {
        // rows g and g + 8 (4 K words on, where no word is the ring's first)
        constexpr int NEXT = OFF + 16 * K;
        const uint32_t w1[2] = {lds<OFF>(at.last), lds<NEXT>(at.last)};
        const uint32_t w0[2] = {lds<OFF>(at.before), lds<NEXT - 4>(at.last)};
        uint32_t w2[2] = {0u, 0u};
        if constexpr (K == 4)
            w2[0] = lds<OFF + 4>(at.last), w2[1] = lds<NEXT + 4>(at.last);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t t = __funnelshift_r(w1[h], w0[h], l.sh);
            if constexpr (K == 1) {        // inputs 2j, 2j + 1, 2j + 8, 2j + 9
                const uint32_t u = t >> 1;
                a[h] = levels2(cut<8>(u), cut<8>(t));
                a[2 + h] = levels2(cut<0>(u), cut<0>(t));
            } else if constexpr (K == 2) { // inputs j, j + 4, j + 8, j + 12
                const uint32_t u = __funnelshift_r(w1[h], w0[h], l.sh + 24);
                a[h] = levels2(cut<0>(u), cut<16>(t));
                a[2 + h] = levels2(cut<8>(t), cut<0>(t));
            } else if constexpr (K == 3) { // inputs 4j .. 4j + 3
                a[h] = levels2(cut<9>(t), cut<6>(t));
                a[2 + h] = levels2(cut<3>(t), cut<0>(t));
            } else {                       // inputs j, j + 4; j + 8, j + 12 end a word later
                const uint32_t u = __funnelshift_r(w2[h], w1[h], l.sh);
                a[h] = levels2(cut<16>(t), cut<0>(t));
                a[2 + h] = levels2(cut<16>(u), cut<0>(u));
            }
        }
    } else {
        // rows 4j .. 4j + 3; two outputs of each.  (Neighbouring rows share words up to K = 2.)
        uint32_t w[4][2], t[4];
        // (up to K = 2 a lane's words from `last` on begin at K * 8 bytes times j)
        if constexpr (K == 1) {
            uint32_t q[3] = {lds<OFF>(at.before)};
            lds2<OFF>(at.last, q[1], q[2]);
#pragma unroll
            for (int r = 0; r < 4; r++)
                t[r] = __funnelshift_r(q[(r >> 1) + 1], q[r >> 1], l.sh - 16 * (r & 1));
        } else if constexpr (K == 2) {
            uint32_t q[5] = {lds<OFF>(at.before)};
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                         : "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]) : "r"(at.last), "n"(OFF));
#pragma unroll
            for (int r = 0; r < 4; r++)
                t[r] = __funnelshift_r(q[r + 1], q[r], l.sh);
        } else if constexpr (K == 3) {
            t[0] = __funnelshift_r(lds<OFF>(at.last), lds<OFF>(at.before), l.sh);
            t[1] = __funnelshift_r(lds<OFF>(at.last1), lds<OFF - 4>(at.last1), l.sh1);
            t[2] = __funnelshift_r(lds<OFF + 12>(at.last), lds<OFF + 8>(at.last), l.sh);
            t[3] = __funnelshift_r(lds<OFF + 12>(at.last1), lds<OFF + 8>(at.last1), l.sh1);
        } else {
            t[0] = __funnelshift_r(lds<OFF>(at.last), lds<OFF>(at.before), l.sh);
            t[1] = __funnelshift_r(lds<OFF + 8>(at.last), lds<OFF + 4>(at.last), l.sh);
            t[2] = __funnelshift_r(lds<OFF + 16>(at.last), lds<OFF + 12>(at.last), l.sh);
            t[3] = __funnelshift_r(lds<OFF + 24>(at.last), lds<OFF + 20>(at.last), l.sh);
        }
#pragma unroll
        for (int r = 0; r < 4; r++) {
            w[r][0] = cut<K == 1 ? 8 : K == 2 ? 16 : K>(t[r]);
            w[r][1] = cut<0>(t[r]);
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

// acc += the products of tiles I .. 3 of a group with their inputs at z: NB * 8 rows of 128
// bytes; those of 8 rows from ANY on are left out where `blocks` says they hold none
template <int K, bool TR, int NB, int ANY, int I = 0>
__device__ __forceinline__ void four_tiles(const Words &at, const Lane &l, uint32_t z, int blocks, float (&acc)[NB][4]) {
    uint32_t f[4];
    fragment<K, TR, I * 32 * K>(at, l, f);
    const uint32_t row = z ^ (uint32_t)(I << 5);
#pragma unroll
    for (int b = 0; b < NB; b++) {
        if (b < ANY || b < blocks) {
            uint32_t b0, b1;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b0), "=r"(b1) : "r"(row + b * 1024u));
            mma16(acc[b], f, b0, b1);
        }
    }
    if constexpr (I < 3)
        four_tiles<K, TR, NB, ANY, I + 1>(at, l, z, blocks, acc);
}

// acc += the products of tiles I .. 7 of a step with their inputs: two panels of 64 inputs,
// PANEL bytes apart, of RB * 8 rows of 128 bytes (LO: and as many of their remainders behind
// them); z[i]: the lane's inputs of tiles i and 4 + i.  Those of 8 rows from the second on
// are left out where `blocks` says they hold none.
template <int K, bool TR, int RB, bool LO, int PANEL, int I = 0, int B = 0>
__device__ __forceinline__ void tile_rows(const uint32_t (&f)[4], uint32_t z, int blocks, float (&acc)[RB][4]) {
    if (B == 0 || B < blocks) {
        constexpr int AT = (I >> 2) * PANEL + B * 1024;
        uint32_t b0, b1;
        lds2<AT>(z, b0, b1);
        mma16(acc[B], f, b0, b1);
        if constexpr (LO) {
            lds2<AT + RB * 1024>(z, b0, b1);
            mma16(acc[B], f, b0, b1);
        }
    }
    if constexpr (B + 1 < RB)
        tile_rows<K, TR, RB, LO, PANEL, I, B + 1>(f, z, blocks, acc);
}
template <int K, bool TR, int RB, bool LO, int PANEL, int I = 0>
__device__ __forceinline__ void eight_tiles(const Words &at, const Lane &l, const uint32_t (&z)[4], int blocks, float (&acc)[RB][4]) {
    uint32_t f[4];
    fragment<K, TR, I * 32 * K>(at, l, f);
    tile_rows<K, TR, RB, LO, PANEL, I>(f, z[I & 3], blocks, acc);
    if constexpr (I < 7)
        eight_tiles<K, TR, RB, LO, PANEL, I + 1>(at, l, z, blocks, acc);
}

}  // namespace exl3
