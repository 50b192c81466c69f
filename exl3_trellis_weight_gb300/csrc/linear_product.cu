// linear_product.cu -- y = z V H . right . 2^-7 s (see linear.cuh), V decoded
// from the codes inside the kernel.  Simple form: one thread per output of a
// block of 128, eight tokens at a time, binary32 sums.
#include "linear.cuh"

namespace exl3 {

namespace {

constexpr int kTok = 8;

template <typename TY>
__global__ void __launch_bounds__(128) product_kernel(const ProductLaunch a) {
    __shared__ float buf[kTok][128];
    const int f0 = blockIdx.x * 128, c = threadIdx.x, e = blockIdx.y;
    const int n_in = (int)(a.transposed ? a.cols : a.rows), n_out = (int)(a.transposed ? a.rows : a.cols);
    const int64_t t_lo = a.offsets ? max(0, a.offsets[e]) : 0;
    const int64_t t_hi = a.offsets ? min((int64_t)a.offsets[e + 1], a.T) : a.T;
    const int64_t NP = act_rows(a.T);
    const int64_t tiles_c = a.cols / 16;
    const uint32_t *codes = a.codes + (size_t)e * (a.rows / 16) * tiles_c * (8 * a.K);
    const float s = a.scale[e] * 0x1p-7f;
    const TY *B = reinterpret_cast<const TY *>(a.B);
    for (int64_t t0 = t_lo + (int64_t)blockIdx.z * kTok; t0 < t_hi; t0 += (int64_t)gridDim.z * kTok) {
        float acc[kTok] = {};
        for (int k = 0; k < n_in; k++) {
            const int64_t r = a.transposed ? f0 + c : k, q = a.transposed ? k : f0 + c;
            const uint32_t *w = codes + (size_t)((r >> 4) * tiles_c + (q >> 4)) * (8 * a.K);
            const float v = mul1_value(window_state_k(w, (int)(r & 15) * 16 + (int)(q & 15), a.K));
#pragma unroll
            for (int i = 0; i < kTok; i++)
                if (t0 + i < t_hi)
                    acc[i] = __fmaf_rn(__half2float(*reinterpret_cast<const __half *>(a.image + act_offset(NP, t0 + i, k))),
                                       v, acc[i]);
        }
#pragma unroll
        for (int i = 0; i < kTok; i++)
            buf[i][c] = acc[i];
        __syncthreads();
        for (int h = 1; h < 128; h <<= 1) {
            float n[kTok];
#pragma unroll
            for (int i = 0; i < kTok; i++)
                n[i] = (c & h) ? buf[i][c ^ h] - buf[i][c] : buf[i][c] + buf[i][c ^ h];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kTok; i++)
                buf[i][c] = n[i];
            __syncthreads();
        }
        for (int i = 0; i < kTok; i++) {
            const int64_t t = t0 + i;
            if (t >= t_hi)
                break;
            float v = buf[i][c] * (a.rscale[t] * s) * a.right[(size_t)e * n_out + f0 + c];
            if (a.B) {
                const int ad = a.slots[t];
                if (ad >= 0 && ad < a.n_adapters) {
                    const int r = a.ranks ? min(max(a.ranks[ad], 0), a.rank) : a.rank;
                    for (int j = 0; j < r; j++)
                        v = __fmaf_rn(a.h[t * a.rank + j], to_f32(B[((size_t)ad * a.rank + j) * n_out + f0 + c]), v);
                }
            }
            reinterpret_cast<TY *>(a.y)[t * a.y_stride + f0 + c] = from_f32<TY>(v);
        }
        __syncthreads();
    }
}

}  // namespace

exl3_status launch_product(const ProductLaunch &p, cudaStream_t s) {
    const int64_t n_out = p.transposed ? p.rows : p.cols;
    const int64_t z = (p.T + kTok - 1) / kTok;
    const dim3 grid((unsigned)(n_out / 128), (unsigned)p.E, (unsigned)(p.offsets ? (z < 8 ? z : 8) : (z < 1024 ? z : 1024)));
    if (p.dt == EXL3_BF16)
        product_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p);
    else
        product_kernel<__half><<<grid, 128, 0, s>>>(p);
    note_launch();
    return cuda_check(cudaGetLastError(), "coded product launch");
}

}  // namespace exl3
