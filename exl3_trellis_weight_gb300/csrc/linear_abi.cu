// linear_abi.cu -- entry points of the products with trellis-coded matrices
// (exl3_linear, exl3_linear_backward, exl3_expert_linear in include/exl3.h):
// argument checks, workspace layout, launch order.
#include "abi_checks.cuh"
#include "linear.cuh"

using namespace exl3;

namespace {

struct Coded {
    const uint16_t *codes;
    int64_t rows, cols;
    int K;
    const float *su, *sv, *scale;
    int transposed;
    int64_t inputs() const { return transposed ? cols : rows; }
    int64_t outputs() const { return transposed ? rows : cols; }
};

bool side_ok(int64_t n) { return n > 0 && n % 128 == 0 && n <= kMaxSide; }

exl3_status check_coded(const Coded &w, int64_t T, int dt) {
    exl3_status st;
    if (dt != EXL3_BF16 && dt != EXL3_F16)
        return set_error(EXL3_ERR_INVALID_ARG, "dtype %d is not EXL3_BF16 or EXL3_F16", dt);
    if (T < 0 || T > kMaxTokens)
        return set_error(EXL3_ERR_INVALID_ARG, "%lld tokens: 0 to 2^24 are supported", (long long)T);
    if (!side_ok(w.rows) || !side_ok(w.cols))
        return set_error(EXL3_ERR_UNSUPPORTED, "rows and cols must be multiples of 128 up to 65536, got %lld x %lld",
                         (long long)w.rows, (long long)w.cols);
    if (!exl3_supports_k(w.K))
        return set_error(EXL3_ERR_UNSUPPORTED, "K=%d is not supported", w.K);
    if ((st = need(w.codes, "codes", 16)) != EXL3_OK) return st;
    if ((st = need(w.su, "su", 16)) != EXL3_OK) return st;
    if ((st = need(w.sv, "sv", 16)) != EXL3_OK) return st;
    return need(w.scale, "scale", 4);
}

struct Adapters {
    const void *A, *B;
    const float *gain;
    const int32_t *slots, *ranks;
    int n, rank;
    int64_t inputs, outputs;  // columns of A and B
};

bool adapters_ok(int n, int rank) { return n >= 0 && n <= kMaxAdapters && (n == 0 || (rank > 0 && rank <= kMaxRank)); }

exl3_status check_adapters(const Adapters &a, int64_t T) {
    exl3_status st;
    if (!adapters_ok(a.n, a.rank))
        return set_error(EXL3_ERR_UNSUPPORTED, "%d adapters of rank %d: at most %d of rank 1 to %d are supported", a.n,
                         a.rank, kMaxAdapters, kMaxRank);
    if (a.n == 0)
        return EXL3_OK;
    if ((st = need(a.A, "A", 16)) != EXL3_OK) return st;
    if ((st = need(a.B, "B", 16)) != EXL3_OK) return st;
    if ((st = need(a.gain, "gain", 4)) != EXL3_OK) return st;
    if (T > 0 && (st = need(a.slots, "slots", 4)) != EXL3_OK) return st;
    if (a.ranks && !aligned(a.ranks, 4))
        return set_error(EXL3_ERR_INVALID_ARG, "ranks is not 4-byte aligned");
    return EXL3_OK;
}

// a result is apart from what the kernels read beside the activations: the codes of E
// matrices and the adapters' factors
exl3_status check_read(const Rows &out, const char *name, const Coded &w, int E, const Adapters &ad) {
    exl3_status st;
    const size_t factors = (size_t)ad.n * ad.rank * 2;
    if ((st = check_apart(out, name, w.codes, (size_t)E * w.rows * w.cols * w.K / 8, "codes")) != EXL3_OK) return st;
    if (ad.n == 0)
        return EXL3_OK;
    if ((st = check_apart(out, name, ad.A, factors * ad.inputs, "A")) != EXL3_OK) return st;
    return check_apart(out, name, ad.B, factors * ad.outputs, "B");
}

// up to here each token's adapter is multiplied on its own (rotation and coded product
// carry it along); with more the tokens are sorted by adapter and multiplied in tiles.
// Both sides, a call in a replayed graph, us, sorted / on its own, 4096 -> 4096, K = 3:
//   4 adapters of rank 16        64 tokens 28.2 / 21.7   96: 30.0 / 23.6   192: 36.6 / 29.4
//   40 adapters of rank 64       64 tokens 38.5 / 30.8   96: 41.9 / 40.4   192: 48.6 / 55.7
//   1000 adapters of rank 16     64 tokens 35.4 / 24.6   96: 42.2 / 28.4   192: 61.6 / 36.6
// On its own a token reads its adapter's factors itself: the sides cross at about 100
// tokens at rank 64 and beyond 192 at rank 16.
constexpr int64_t kFewTokens = 64;

struct LinearWs {
    unsigned char *image;     // rotated activations
    float *rscale;            // [T]
    float *h, *g;             // [T][rank]: x A^T and, for the gradient, dy B^T
    int32_t *plan;            // tokens by adapter
    float *term;              // [T][outputs]: the adapters' part of the result
    size_t bytes;
    LinearWs(void *ws, int64_t T, int64_t inputs, int64_t outputs, int n, int rank, bool grad) {
        Carve c{(unsigned char *)ws};
        image = c.take<unsigned char>((size_t)act_rows(T) * inputs * 2);
        rscale = c.take<float>((size_t)T);
        h = n ? c.take<float>((size_t)T * rank) : nullptr;
        g = n && grad ? c.take<float>((size_t)T * rank) : nullptr;
        plan = n ? c.take<int32_t>(adapt_plan_ints(T, n)) : nullptr;
        term = n && T > kFewTokens ? c.take<float>((size_t)T * outputs) : nullptr;
        bytes = c.used;
        // one workspace of the gradients' size serves both directions of a layer
        if (grad) {
            const size_t forward = LinearWs(nullptr, T, outputs, inputs, n, rank, false).bytes;
            bytes = bytes > forward ? bytes : forward;
        }
    }
};

// y = x W^ (or its transpose), adapters' rank-sided products in h added with B.
// beside: kernels of the same call run already (plan and shrink), the rotation runs
// beside them (they are latency, it is instructions); back: the adapters' way back, to
// m.term, comes between it and the product.
exl3_status run_linear(const LinearWs &m, const void *x, int dt, int64_t T, int64_t x_stride, const Coded &w, int E,
                       const int32_t *offsets, const void *A, const void *B, float *h, const Adapters &ad, void *y,
                       int64_t y_stride, cudaStream_t s, bool beside = false, const AdaptLaunch *back = nullptr) {
    exl3_status st;
    PrepLaunch a = {};
    a.x = x;
    a.dt = dt;
    a.T = T;
    a.stride = x_stride;
    a.n = (int)w.inputs();
    a.left = w.transposed ? w.sv : w.su;
    a.offsets = offsets;
    a.E = E;
    a.image = m.image;
    a.rscale = m.rscale;
    a.y = y;
    a.y_stride = y_stride;
    a.y_cols = (int)w.outputs();
    a.M = A;
    a.gain = ad.gain;
    a.slots = ad.slots;
    a.ranks = ad.ranks;
    a.n_adapters = A ? ad.n : 0;
    a.rank = ad.rank;
    a.h = h;
    a.beside = beside;
    ProductLaunch p = {};
    p.image = m.image;
    p.rscale = m.rscale;
    p.T = T;
    p.codes = reinterpret_cast<const uint32_t *>(w.codes);
    p.rows = w.rows;
    p.cols = w.cols;
    p.K = w.K;
    p.right = w.transposed ? w.su : w.sv;
    p.scale = w.scale;
    p.transposed = w.transposed;
    p.offsets = offsets;
    p.E = E;
    p.B = B;
    p.h = h;
    p.term = back ? m.term : nullptr;
    p.slots = ad.slots;
    p.ranks = ad.ranks;
    p.n_adapters = ad.n;
    p.rank = ad.rank;
    p.y = y;
    p.dt = dt;
    p.y_stride = y_stride;
    const bool few = few_eligible(p);
    a.order = few ? few_order(p) : 0;
    if ((st = launch_prep(a, s)) != EXL3_OK) return st;
    if (back && (st = launch_expand(*back, m.term, s)) != EXL3_OK) return st;
    return few ? launch_product_few(p, s) : launch_product(p, s);
}

AdaptLaunch adapt_of(const LinearWs &m, int dt, int64_t T, const Adapters &ad) {
    AdaptLaunch p = {};
    p.plan = adapt_plan(m.plan, T, ad.n);
    p.dt = dt;
    p.T = T;
    p.n = ad.n;
    p.rank = ad.rank;
    p.gain = ad.gain;
    p.slots = ad.slots;
    p.ranks = ad.ranks;
    return p;
}

bool sizes_ok(int64_t T, int64_t rows, int64_t cols, int n, int rank) {
    return T >= 0 && T <= kMaxTokens && side_ok(rows) && side_ok(cols) && adapters_ok(n, rank);
}

}  // namespace

extern "C" {

size_t exl3_linear_workspace_bytes(int64_t T, int64_t rows, int64_t cols, int transposed, int n_adapters, int rank) {
    if (!sizes_ok(T, rows, cols, n_adapters, rank))
        return 0;
    return LinearWs(nullptr, T, transposed ? cols : rows, transposed ? rows : cols, n_adapters, rank, false).bytes;
}

exl3_status exl3_linear(const void *x, int dt, int64_t T, int64_t x_stride, const uint16_t *codes, int64_t rows,
                        int64_t cols, int K, const float *su, const float *sv, const float *scale, int transposed,
                        const void *A, const void *B, const float *gain, const int32_t *slots, const int32_t *ranks,
                        int n_adapters, int rank, void *y, int64_t y_stride, void *ws, size_t ws_bytes, void *stream) {
    exl3_status st;
    const Coded w{codes, rows, cols, K, su, sv, scale, transposed ? 1 : 0};
    const Adapters ad{A, B, gain, slots, ranks, n_adapters, rank, w.inputs(), w.outputs()};
    if ((st = check_coded(w, T, dt)) != EXL3_OK) return st;
    if ((st = check_adapters(ad, T)) != EXL3_OK) return st;
    const Rows xr{x, T, w.inputs(), x_stride}, yr{y, T, w.outputs(), y_stride};
    if ((st = check_rows(xr, "x")) != EXL3_OK) return st;
    if ((st = check_rows(yr, "y")) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", xr, "x")) != EXL3_OK) return st;
    if ((st = check_read(yr, "y", w, 1, ad)) != EXL3_OK) return st;
    if (T == 0)
        return EXL3_OK;
    const LinearWs m(ws, T, w.inputs(), w.outputs(), n_adapters, rank, false);
    if ((st = check_ws(ws, ws_bytes, m.bytes)) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", ws, m.bytes, "the workspace")) != EXL3_OK) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (n_adapters && T > kFewTokens) {
        AdaptLaunch p = adapt_of(m, dt, T, ad);
        p.side[0] = {x, x_stride, (int)w.inputs(), A, m.h, p.plan.largest, nullptr};
        if ((st = launch_adapt_plan(p, s)) != EXL3_OK) return st;
        if ((st = launch_shrink(p, 1, s)) != EXL3_OK) return st;
        p.side[0].M = B;
        p.side[0].n = (int)w.outputs();
        return run_linear(m, x, dt, T, x_stride, w, 1, nullptr, nullptr, nullptr, nullptr, ad, y, y_stride, s, true, &p);
    }
    return run_linear(m, x, dt, T, x_stride, w, 1, nullptr, A, n_adapters ? B : nullptr, m.h, ad, y, y_stride, s);
}

size_t exl3_linear_backward_workspace_bytes(int64_t T, int64_t rows, int64_t cols, int transposed, int n_adapters,
                                            int rank) {
    if (!sizes_ok(T, rows, cols, n_adapters, rank))
        return 0;
    return LinearWs(nullptr, T, transposed ? rows : cols, transposed ? cols : rows, n_adapters, rank, true).bytes;
}

exl3_status exl3_linear_backward(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, int dt, int64_t T,
                                 const uint16_t *codes, int64_t rows, int64_t cols, int K, const float *su,
                                 const float *sv, const float *scale, int transposed, const void *A, const void *B,
                                 const float *gain, const int32_t *slots, const int32_t *ranks, int n_adapters,
                                 int rank, void *dx, int64_t dx_stride, void *dA, void *dB, void *ws,
                                 size_t ws_bytes, void *stream) {
    exl3_status st;
    // the gradient of x is a product with the other transposition
    const Coded w{codes, rows, cols, K, su, sv, scale, transposed ? 0 : 1};
    // (w's outputs are the forward product's inputs)
    const Adapters ad{A, B, gain, slots, ranks, n_adapters, rank, w.outputs(), w.inputs()};
    if ((st = check_coded(w, T, dt)) != EXL3_OK) return st;
    if ((st = check_adapters(ad, T)) != EXL3_OK) return st;
    const int64_t n_in = w.outputs(), n_out = w.inputs();      // of the forward product
    const Rows dyr{dy, T, n_out, dy_stride}, xr{x, T, n_in, x_stride}, dxr{dx, T, n_in, dx_stride};
    if ((st = check_rows(dyr, "dy")) != EXL3_OK) return st;
    if ((st = check_rows(dxr, "dx")) != EXL3_OK) return st;
    if (n_adapters) {
        if ((st = check_rows(xr, "x")) != EXL3_OK) return st;
        if ((st = need(dA, "dA", 16)) != EXL3_OK) return st;
        if ((st = need(dB, "dB", 16)) != EXL3_OK) return st;
        if ((st = check_apart(dxr, "dx", xr, "x")) != EXL3_OK) return st;
    }
    if ((st = check_apart(dxr, "dx", dyr, "dy")) != EXL3_OK) return st;
    if ((st = check_read(dxr, "dx", w, 1, ad)) != EXL3_OK) return st;
    // dA and dB are written beside the product, while x and dy are read
    const int64_t factors = (int64_t)n_adapters * rank;
    const Rows dAr{dA, n_adapters ? 1 : 0, factors * n_in, factors * n_in}, dBr{dB, n_adapters ? 1 : 0, factors * n_out, factors * n_out};
    for (int k = 0; k < 2; k++) {
        const Rows &d = k ? dBr : dAr;
        const char *name = k ? "dB" : "dA";
        if ((st = check_read(d, name, w, 1, ad)) != EXL3_OK) return st;
        if ((st = check_apart(d, name, x, xr.bytes(), "x")) != EXL3_OK) return st;
        if ((st = check_apart(d, name, dy, dyr.bytes(), "dy")) != EXL3_OK) return st;
        if ((st = check_apart(d, name, dx, dxr.bytes(), "dx")) != EXL3_OK) return st;
    }
    if ((st = check_apart(dAr, "dA", dB, dBr.bytes(), "dB")) != EXL3_OK) return st;
    if (T == 0 && n_adapters == 0)
        return EXL3_OK;
    const LinearWs m(ws, T, n_out, n_in, n_adapters, rank, true);
    if ((st = check_ws(ws, ws_bytes, m.bytes)) != EXL3_OK) return st;
    if ((st = check_apart(dxr, "dx", ws, m.bytes, "the workspace")) != EXL3_OK) return st;
    if ((st = check_apart(dAr, "dA", ws, m.bytes, "the workspace")) != EXL3_OK) return st;
    if ((st = check_apart(dBr, "dB", ws, m.bytes, "the workspace")) != EXL3_OK) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (n_adapters == 0)
        return run_linear(m, dy, dt, T, dy_stride, w, 1, nullptr, nullptr, nullptr, nullptr, ad, dx, dx_stride, s);
    AdaptLaunch p = adapt_of(m, dt, T, ad);
    p.side[0] = {x, x_stride, (int)n_in, A, m.h, p.plan.largest, dA};
    p.side[1] = {dy, dy_stride, (int)n_out, B, m.g, p.plan.largest + ad.n, dB};
    if ((st = launch_adapt_plan(p, s)) != EXL3_OK) return st;
    if (T) {
        if ((st = launch_shrink(p, 2, s)) != EXL3_OK) return st;
        AdaptLaunch q = p;
        q.side[0] = {nullptr, 0, (int)n_in, A, m.g, nullptr, nullptr};
        const bool few = T <= kFewTokens;                 // the coded product adds the adapters' terms itself
        if ((st = run_linear(m, dy, dt, T, dy_stride, w, 1, nullptr, nullptr, few ? A : nullptr, few ? m.g : nullptr, ad,
                             dx, dx_stride, s, true, few ? nullptr : &q)) != EXL3_OK)
            return st;
    }
    // dA = sum g x^T, dB = sum h dy^T, beside the product's end
    p.side[0].h = m.g;
    p.side[0].largest = p.plan.largest + ad.n;
    p.side[1].h = m.h;
    p.side[1].largest = p.plan.largest;
    return launch_outer(p, s);
}

size_t exl3_expert_linear_workspace_bytes(int64_t T, int64_t rows, int64_t cols, int transposed) {
    return exl3_linear_workspace_bytes(T, rows, cols, transposed, 0, 0);
}

exl3_status exl3_expert_linear(const void *x, int dt, int64_t T, int64_t x_stride, const int32_t *offsets,
                               int n_experts, const uint16_t *codes, int64_t rows, int64_t cols, int K,
                               const float *su, const float *sv, const float *scale, int transposed, void *y,
                               int64_t y_stride, void *ws, size_t ws_bytes, void *stream) {
    exl3_status st;
    const Coded w{codes, rows, cols, K, su, sv, scale, transposed ? 1 : 0};
    if ((st = check_coded(w, T, dt)) != EXL3_OK) return st;
    if (n_experts < 1 || n_experts > kMaxExperts)
        return set_error(EXL3_ERR_UNSUPPORTED, "%d experts: 1 to %d are supported", n_experts, kMaxExperts);
    if ((st = need(offsets, "offsets", 4)) != EXL3_OK) return st;
    const Rows xr{x, T, w.inputs(), x_stride}, yr{y, T, w.outputs(), y_stride};
    if ((st = check_rows(xr, "x")) != EXL3_OK) return st;
    if ((st = check_rows(yr, "y")) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", xr, "x")) != EXL3_OK) return st;
    if ((st = check_read(yr, "y", w, n_experts, Adapters{})) != EXL3_OK) return st;
    if (T == 0)
        return EXL3_OK;
    const LinearWs m(ws, T, w.inputs(), w.outputs(), 0, 0, false);
    if ((st = check_ws(ws, ws_bytes, m.bytes)) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", ws, m.bytes, "the workspace")) != EXL3_OK) return st;
    return run_linear(m, x, dt, T, x_stride, w, n_experts, offsets, nullptr, nullptr, nullptr, Adapters{}, y, y_stride,
                      (cudaStream_t)stream);
}

}  // extern "C"
