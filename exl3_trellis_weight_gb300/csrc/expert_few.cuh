// expert_few.cuh -- the sums of an expert's few rows with a coded matrix, as in
// linear_few.cu: a warp owns 16 outputs, its tiles of codes arrive in a ring and become
// A fragments, the rotated activations of the block's inputs lie in shared memory.
#pragma once

#include "layer.cuh"
#include "linear_few.cuh"

namespace exl3 {

constexpr int kExpertWarps = 16, kExpertThreads = kExpertWarps * 32;

template <int K> struct CodeRing {
    static constexpr int kLanes = 2 * K, kAtOnce = 4;         // lanes of a tile; tiles of a copy group
    static constexpr uint32_t kBytes = kTilesAhead * 32 * K;  // of a warp
    static_assert(kLanes * kAtOnce <= 32 && kTilesAhead % kAtOnce == 0, "one copy group is one instruction");
    uint32_t ring, dst;
    const char *src;
    int64_t hop;
    int q_lo, q_hi;
    bool mine;

    // tiles q_lo .. q_hi - 1 of 16 inputs from `codes` on, `hop` bytes apart
    __device__ __forceinline__ CodeRing(uint32_t at, const void *codes, int64_t hop_, int lo, int hi, int lane)
        : ring(at), dst(at + (uint32_t)lane * 16), hop(hop_), q_lo(lo), q_hi(hi), mine(lane < kLanes * kAtOnce) {
        src = reinterpret_cast<const char *>(codes) + (lane / kLanes) * hop + (lane % kLanes) * 16;
    }
    __device__ __forceinline__ void load(int q) const {
        if (mine && q < q_hi)
            tc::copy16(dst + (uint32_t)((q - q_lo) % kTilesAhead) * (32 * K), src + (int64_t)q * hop);
        tc::copy_group();
    }
    __device__ __forceinline__ void begin() const {
#pragma unroll
        for (int i = 0; i < kTilesAhead; i += kAtOnce)
            load(q_lo + i);
    }
};

// acc += the tiles' products; z: shared memory of the rows' inputs, 64 inputs of NB * 8
// rows a block of NB * 1024 bytes, from the block of tile 0 on; `blocks` of 8 rows hold any
template <int K, bool TR, int NB>
__device__ __forceinline__ void few_sums(const CodeRing<K> &r, uint32_t z0, int blocks, int lane, float (&acc)[NB][4]) {
    const int g = lane >> 2, j = lane & 3;
    const Lane l = lane_of<K, TR>(g, j);
    uint32_t tiles = r.ring;
    // row g's four inputs of tile i: 8 bytes of chunk 2 i + j / 2 of its row
    uint32_t z = z0 + (uint32_t)(r.q_lo >> 2) * (NB * 1024u) + (uint32_t)g * 128u + ((uint32_t)((j >> 1) ^ g) << 4) + (uint32_t)(j & 1) * 8u;
    for (int q = r.q_lo; q < r.q_hi; q += CodeRing<K>::kAtOnce, z += NB * 1024u) {
        tc::copy_wait<kTilesAhead / CodeRing<K>::kAtOnce - 1>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < CodeRing<K>::kAtOnce; i++) {
            uint32_t f[4];
            fragment<K, TR>(tiles + i * (32 * K), l, f);
            const uint32_t row = z ^ (uint32_t)(i << 5);
#pragma unroll
            for (int b = 0; b < NB; b++) {
                if (NB <= 2 || b < blocks) {
                    uint32_t b0, b1;
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b0), "=r"(b1) : "r"(row + b * 1024u));
                    mma16(acc[b], f, b0, b1);
                }
            }
        }
        __syncwarp();                      // every lane has read the tiles that the next copies replace
        r.load(q + kTilesAhead);
        tiles += CodeRing<K>::kAtOnce * 32 * K;
        if (tiles == r.ring + CodeRing<K>::kBytes)
            tiles = r.ring;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// a warp's sums to [row][128 outputs], float4 f of a row at out_at(f)
template <int K, bool TR, int NB>
__device__ __forceinline__ void put_sums(float *sums, const float (&acc)[NB][4], int fw, int lane, const float *factor) {
    const int g = lane >> 2, j = lane & 3;
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int o = fw * 16 + (TR || K <= 2 ? g + 8 * (i >> 1) : 2 * g + (i >> 1)), t = b * 8 + 2 * j + (i & 1);
            sums[t * 128 + 4 * out_at(o >> 2) + (o & 3)] = factor ? __fmul_rn(acc[b][i], factor[t]) : acc[b][i];
        }
}

// Blocks of a cluster that share the inputs of a tile, and shared memory: blocks that would
// idle (two fit an SM) take shares of at least 128 inputs each; false where the activations
// of a share do not fit.
struct ExpertShape {
    int split;
    uint32_t ring_off, smem;
};
inline bool expert_shape(ExpertShape &f, int64_t tiles, int n_in, int tile_n, int K, int matrices, int64_t sms) {
    const int steps = n_in / 128;
    const uint32_t sums = 2u * (uint32_t)tile_n * 512u, ring = (uint32_t)kExpertWarps * kTilesAhead * 32u * (uint32_t)K;
    auto z_bytes = [&](int split) {
        const uint32_t z = (uint32_t)((steps + split - 1) / split) * (uint32_t)tile_n * 256u * (uint32_t)matrices;
        return z > sums ? z : sums;
    };
    f.split = 1;
    while (f.split < 8 && steps >= f.split * 2 && (tiles * f.split * 2 <= 2 * sms || z_bytes(f.split) + ring > 100u * 1024u))
        f.split *= 2;
    f.ring_off = z_bytes(f.split);
    f.smem = f.ring_off + ring + 1024u;
    return f.smem <= 220u * 1024u;
}

}  // namespace exl3
