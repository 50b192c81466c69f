// layer_abi.cu -- entry points of what stands around the coded products of a layer
// (exl3_rms_norm, exl3_rms_norm_backward, exl3_quantize8, exl3_linear8,
// exl3_expert_layer in include/exl3.h): argument checks, workspace layout, launch order.
#include "abi_checks.cuh"
#include "layer.cuh"

using namespace exl3;

namespace {

exl3_status check_16bit(int dt) {
    if (dt != EXL3_BF16 && dt != EXL3_F16)
        return set_error(EXL3_ERR_INVALID_ARG, "dtype %d is not EXL3_BF16 or EXL3_F16", dt);
    return EXL3_OK;
}

exl3_status check_tokens(int64_t T) {
    if (T < 0 || T > kMaxTokens)
        return set_error(EXL3_ERR_INVALID_ARG, "%lld tokens: 0 to 2^24 are supported", (long long)T);
    return EXL3_OK;
}

int64_t blocks_of(int64_t n) { return (n + 127) / 128; }

// an output may be an input itself (each thread reads its columns before it writes them),
// or apart from it
exl3_status check_same_or_apart(const Rows &out, const char *name, const Rows &r, const char *other) {
    if (out.p == r.p && (out.stride == r.stride || out.T <= 1))
        return EXL3_OK;
    return check_apart(out, name, r, other);
}

bool norm_ok(int64_t T, int64_t n) { return T >= 0 && T <= kMaxTokens && n >= 1 && n <= kMaxNorm; }

exl3_status check_norm(int dt, int64_t T, int64_t n, const void *weight, int w_dt, float eps) {
    exl3_status st;
    // (a normal number is above what the squares of a row lose below binary32's range)
    if (!(eps >= 0x1p-126f && eps <= 0x1.fffffep127f))
        return set_error(EXL3_ERR_INVALID_ARG, "eps = %g is not a positive normal number", (double)eps);
    if ((st = check_16bit(dt)) != EXL3_OK) return st;
    if ((st = check_tokens(T)) != EXL3_OK) return st;
    if (!norm_ok(T, n))
        return set_error(EXL3_ERR_UNSUPPORTED, "norm of %lld columns: 1 to %lld are supported", (long long)n, (long long)kMaxNorm);
    if (w_dt != dt && w_dt != EXL3_F32)
        return set_error(EXL3_ERR_INVALID_ARG, "weight's dtype %d is neither the rows' nor EXL3_F32", w_dt);
    return need(weight, "weight", w_dt == EXL3_F32 ? 4 : 2);
}

bool linear8_ok(int64_t T, int64_t rows, int64_t cols) {
    return T >= 0 && T <= kMaxTokens && rows > 0 && cols > 0 && rows % 16 == 0 && cols % 16 == 0 && rows <= kMaxSide && cols <= kMaxSide;
}

struct Linear8Ws {
    uint8_t *codes;           // x in e4m3
    float *scale;             // [blocks][T]
    size_t bytes;
    Linear8Ws(void *ws, int64_t T, int64_t n_in) {
        Carve c{(unsigned char *)ws};
        codes = c.take<uint8_t>((size_t)(T * n_in));
        scale = c.take<float>((size_t)(T * blocks_of(n_in)));
        bytes = c.used;
    }
};

// Up to 256 tokens.  A call, and the same of router, sort, three exl3_expert_linear and the sum (in
// brackets the three products alone), replayed graphs, us, 64 experts 2048 / 1024, 8 picks, K = 2:
//   tokens      64               128              192              256
//   bfloat16    156 / 284 (196)  206 / 305 (208)  241 / 324 (215)  306 / 339 (219)
//   float16     184 / 281 (194)  261 / 303 (205)  344 / 324 (216)  434 / 339 (220)
// (K = 4: 172, 225, 263 and 331; 203, 287, 380 and 479.)  In float16 the parts are faster from about 170
// tokens on here, where an expert has 20 rows; with more experts it is later.
constexpr int kMaxPicks = 32;
constexpr int64_t kMaxLayerTokens = 256, kMaxPairs = 4096, kMaxLayerSide = 32768;

bool layer_side(int64_t n) { return n > 0 && n % 128 == 0 && n <= kMaxLayerSide; }

bool layer_ok(int64_t T, int64_t H, int64_t F, int E, int top_k) {
    return T >= 0 && T <= kMaxLayerTokens && layer_side(H) && layer_side(F) && E >= 1 && E <= kMaxExperts && top_k >= 1 &&
           top_k <= kMaxPicks && top_k <= E && T * top_k <= kMaxPairs;
}

// pointers of the workspace; the picks are in it unless they are given
size_t carve_layer(ExpertLaunch &p, void *ws) {
    Carve c{(unsigned char *)ws};
    const int64_t n = p.T * p.top_k;
    p.rows = expert_rows(p.T, p.top_k, p.E);
    p.logits = c.take<float>((size_t)(p.T * p.E));
    int32_t *ids = c.take<int32_t>((size_t)n);
    float *weights = c.take<float>((size_t)n);
    if (p.router || !p.ids) {
        p.ids = ids;
        p.weights = weights;
    }
    p.pair_of = c.take<int32_t>((size_t)p.rows);
    // (the size is the same for both types of x)
    const int least = expert_tile_n(p.T, p.top_k, p.E, true), most = expert_tile_n(p.T, p.top_k, p.E, false);
    p.tile_n = p.dt == EXL3_F16 ? least : most;
    const size_t tiles = (size_t)expert_tiles(p.T, p.top_k, p.E, least);
    p.tiles = c.take<int4>(tiles);
    p.up_done = c.take<int32_t>(tiles * (p.F / 128));
    p.down_done = c.take<int32_t>(tiles * (p.H / 128));
    p.sums = c.take<float>((size_t)expert_blocks() * 4 * most * 128);
    p.n_tiles = c.take<int32_t>(1);
    for (int w = 0; w < 2; w++) {
        p.image[w] = c.take<unsigned char>((size_t)act_rows(p.rows) * p.H * 4);
        p.rscale[w] = c.take<float>((size_t)p.rows);
    }
    p.inner = c.take<unsigned char>((size_t)act_rows(p.rows) * p.F * 4);
    p.inner_scale = c.take<float>((size_t)(p.rows * (p.F / 128)));
    p.part = c.take<float>((size_t)n * p.H);
    return c.used;
}

}  // namespace

extern "C" {

exl3_status exl3_rms_norm(const void *x, int dt, int64_t T, int64_t n, int64_t x_stride, const void *residual,
                          int64_t r_stride, const void *weight, int w_dt, float eps, void *h, int64_t h_stride, void *y,
                          int64_t y_stride, uint8_t *y8, float *scale, void *stream) {
    exl3_status st;
    if ((st = check_norm(dt, T, n, weight, w_dt, eps)) != EXL3_OK) return st;
    if (T == 0)
        return EXL3_OK;
    if (!y && !y8)
        return set_error(EXL3_ERR_INVALID_ARG, "neither y nor y8 is there");
    if (!y8 != !scale)
        return set_error(EXL3_ERR_INVALID_ARG, "y8 and scale go together");
    if (scale && !aligned(scale, 4))
        return set_error(EXL3_ERR_INVALID_ARG, "scale is not 4-byte aligned");
    const Rows xr{x, T, n, x_stride}, rr{residual, T, n, r_stride}, hr{residual ? h : nullptr, residual ? T : 0, n, h_stride};
    const Rows yr{y, y ? T : 0, n, y_stride}, qr{y8, y8 ? T : 0, n, n, 1}, sr{scale, y8 ? blocks_of(n) : 0, T, T, 4};
    const size_t w_bytes = (size_t)n * (w_dt == EXL3_F32 ? 4 : 2);
    if ((st = check_rows(xr, "x")) != EXL3_OK) return st;
    if (residual) {
        if ((st = check_rows(rr, "residual")) != EXL3_OK) return st;
        if ((st = check_rows(hr, "h")) != EXL3_OK) return st;
        if ((st = check_same_or_apart(hr, "h", xr, "x")) != EXL3_OK) return st;
        if ((st = check_same_or_apart(hr, "h", rr, "residual")) != EXL3_OK) return st;
        if ((st = check_apart(hr, "h", weight, w_bytes, "weight")) != EXL3_OK) return st;
    }
    if (y) {
        if ((st = check_rows(yr, "y")) != EXL3_OK) return st;
        if ((st = check_same_or_apart(yr, "y", xr, "x")) != EXL3_OK) return st;
        if (residual && (st = check_apart(yr, "y", rr, "residual")) != EXL3_OK) return st;
        if (residual && (st = check_apart(yr, "y", hr, "h")) != EXL3_OK) return st;
        if ((st = check_apart(yr, "y", weight, w_bytes, "weight")) != EXL3_OK) return st;
    }
    for (int k = 0; k < 2 && y8; k++) {
        const Rows &o = k ? sr : qr;
        const char *name = k ? "scale" : "y8";
        if ((st = check_apart(o, name, x, xr.bytes(), "x")) != EXL3_OK) return st;
        if (residual && (st = check_apart(o, name, residual, rr.bytes(), "residual")) != EXL3_OK) return st;
        if (residual && (st = check_apart(o, name, h, hr.bytes(), "h")) != EXL3_OK) return st;
        if ((st = check_apart(o, name, y, yr.bytes(), "y")) != EXL3_OK) return st;
        if ((st = check_apart(o, name, weight, w_bytes, "weight")) != EXL3_OK) return st;
    }
    if (y8 && (st = check_apart(qr, "y8", scale, sr.bytes(), "scale")) != EXL3_OK) return st;
    NormLaunch p = {};
    p.x = x;
    p.residual = residual;
    p.x_stride = x_stride;
    p.r_stride = r_stride;
    p.dt = dt;
    p.T = T;
    p.n = (int)n;
    p.weight = weight;
    p.w_dt = w_dt;
    p.eps = eps;
    p.h = h;
    p.h_stride = h_stride;
    p.y = y;
    p.y_stride = y_stride;
    p.y8 = y8;
    p.scale = scale;
    return launch_norm(p, (cudaStream_t)stream);
}

size_t exl3_rms_norm_backward_workspace_bytes(int64_t T, int64_t n) {
    if (!norm_ok(T, n))
        return 0;
    const size_t parts = (size_t)(norm_grad_parts(T, n) * n) * sizeof(float);
    return align_up(parts ? parts : 1, kAlign);
}

exl3_status exl3_rms_norm_backward(const void *dy, int64_t dy_stride, const void *h, int64_t h_stride, int dt, int64_t T,
                                   int64_t n, const void *weight, int w_dt, float eps, const void *dh, int64_t dh_stride,
                                   void *dx, int64_t dx_stride, void *dweight, void *ws, size_t ws_bytes, void *stream) {
    exl3_status st;
    if ((st = check_norm(dt, T, n, weight, w_dt, eps)) != EXL3_OK) return st;
    const size_t w_size = w_dt == EXL3_F32 ? 4 : 2, w_bytes = (size_t)n * w_size;
    const Rows dyr{dy, T, n, dy_stride}, hr{h, T, n, h_stride}, dhr{dh, dh ? T : 0, n, dh_stride}, dxr{dx, T, n, dx_stride};
    if ((st = check_rows(dyr, "dy")) != EXL3_OK) return st;
    if ((st = check_rows(hr, "h")) != EXL3_OK) return st;
    if ((st = check_rows(dhr, "dh")) != EXL3_OK) return st;
    if ((st = check_rows(dxr, "dx")) != EXL3_OK) return st;
    if ((st = check_same_or_apart(dxr, "dx", dyr, "dy")) != EXL3_OK) return st;
    if ((st = check_apart(dxr, "dx", hr, "h")) != EXL3_OK) return st;
    if (dh && (st = check_same_or_apart(dxr, "dx", dhr, "dh")) != EXL3_OK) return st;
    if ((st = check_apart(dxr, "dx", weight, w_bytes, "weight")) != EXL3_OK) return st;
    NormGradLaunch p = {};
    if (dweight) {
        if ((st = need(dweight, "dweight", w_size)) != EXL3_OK) return st;
        const Rows dwr{dweight, 1, n, n, (int)w_size};
        if ((st = check_apart(dwr, "dweight", dy, dyr.bytes(), "dy")) != EXL3_OK) return st;
        if ((st = check_apart(dwr, "dweight", h, hr.bytes(), "h")) != EXL3_OK) return st;
        if ((st = check_apart(dwr, "dweight", dh, dhr.bytes(), "dh")) != EXL3_OK) return st;
        if ((st = check_apart(dwr, "dweight", dx, dxr.bytes(), "dx")) != EXL3_OK) return st;
        if ((st = check_apart(dwr, "dweight", weight, w_bytes, "weight")) != EXL3_OK) return st;
        const size_t want = exl3_rms_norm_backward_workspace_bytes(T, n);
        if ((st = check_ws(ws, ws_bytes, want)) != EXL3_OK) return st;
        if ((st = check_apart(dwr, "dweight", ws, want, "the workspace")) != EXL3_OK) return st;
        if ((st = check_apart(dxr, "dx", ws, want, "the workspace")) != EXL3_OK) return st;
    }
    p.dy = dy;
    p.h = h;
    p.dh = dh;
    p.dy_stride = dy_stride;
    p.h_stride = h_stride;
    p.dh_stride = dh_stride;
    p.dt = dt;
    p.T = T;
    p.n = (int)n;
    p.weight = weight;
    p.w_dt = w_dt;
    p.eps = eps;
    p.dx = dx;
    p.dx_stride = dx_stride;
    p.dweight = dweight;
    p.part = reinterpret_cast<float *>(ws);
    return launch_norm_grad(p, (cudaStream_t)stream);
}

exl3_status exl3_quantize8(const void *x, int dt, int64_t T, int64_t n, int64_t x_stride, int block_rows, uint8_t *codes,
                           float *scale, void *stream) {
    exl3_status st;
    if (dt != EXL3_F32 && (st = check_16bit(dt)) != EXL3_OK) return st;
    if ((st = check_tokens(T)) != EXL3_OK) return st;
    if (n < 1 || n > kMaxSide)
        return set_error(EXL3_ERR_UNSUPPORTED, "%lld columns: 1 to %lld are supported", (long long)n, (long long)kMaxSide);
    if (block_rows != 1 && block_rows != 128)
        return set_error(EXL3_ERR_UNSUPPORTED, "blocks of %d rows: 1 and 128 are supported", block_rows);
    const Rows xr{x, T, n, x_stride, dt == EXL3_F32 ? 4 : 2}, qr{codes, T, n, n, 1};
    const Rows sr{scale, T ? 1 : 0, (block_rows == 1 ? T : blocks_of(T)) * blocks_of(n), (block_rows == 1 ? T : blocks_of(T)) * blocks_of(n), 4};
    if ((st = check_rows(xr, "x")) != EXL3_OK) return st;
    if (T == 0)
        return EXL3_OK;
    if ((st = need(codes, "codes", 1)) != EXL3_OK) return st;
    if ((st = need(scale, "scale", 4)) != EXL3_OK) return st;
    if ((st = check_apart(qr, "codes", x, xr.bytes(), "x")) != EXL3_OK) return st;
    if ((st = check_apart(sr, "scale", x, xr.bytes(), "x")) != EXL3_OK) return st;
    if ((st = check_apart(qr, "codes", scale, sr.bytes(), "scale")) != EXL3_OK) return st;
    return launch_quantize8({x, dt, T, n, x_stride, block_rows, codes, scale}, (cudaStream_t)stream);
}

size_t exl3_linear8_workspace_bytes(int64_t T, int64_t rows, int64_t cols, int transposed) {
    if (!linear8_ok(T, rows, cols))
        return 0;
    const size_t bytes = Linear8Ws(nullptr, T, transposed ? cols : rows).bytes;
    return bytes ? bytes : kAlign;
}

exl3_status exl3_linear8(const void *x, int x_dt, int64_t T, int64_t x_stride, const float *x_scale, int64_t xs_t,
                         int64_t xs_b, const uint8_t *w, const float *w_scale, int64_t rows, int64_t cols, int transposed,
                         void *y, int y_dt, int64_t y_stride, void *ws, size_t ws_bytes, void *stream) {
    exl3_status st;
    const bool coded = x_dt == EXL3_E4M3;
    if (!coded && (st = check_16bit(x_dt)) != EXL3_OK) return st;
    if ((st = check_16bit(y_dt)) != EXL3_OK) return st;
    if ((st = check_tokens(T)) != EXL3_OK) return st;
    if (!linear8_ok(T, rows, cols))
        return set_error(EXL3_ERR_UNSUPPORTED, "rows and cols must be multiples of 16 up to 65536, got %lld x %lld",
                         (long long)rows, (long long)cols);
    const int64_t n_in = transposed ? cols : rows, n_out = transposed ? rows : cols;
    if ((st = need(w, "w", 16)) != EXL3_OK) return st;
    if ((st = need(w_scale, "w_scale", 4)) != EXL3_OK) return st;
    const Rows xr{x, T, n_in, x_stride, coded ? 1 : 2}, yr{y, T, n_out, y_stride};
    if ((st = check_rows(xr, "x")) != EXL3_OK) return st;
    if ((st = check_rows(yr, "y")) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", xr, "x")) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", w, (size_t)(rows * cols), "w")) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", w_scale, (size_t)(blocks_of(rows) * blocks_of(cols)) * 4, "w_scale")) != EXL3_OK) return st;
    if (!coded && x_scale)
        return set_error(EXL3_ERR_INVALID_ARG, "x_scale goes with x in EXL3_E4M3");
    if (T == 0)
        return EXL3_OK;
    Linear8Launch p = {};
    p.T = T;
    p.w = w;
    p.rows = rows;
    p.cols = cols;
    p.ws = w_scale;
    p.transposed = transposed ? 1 : 0;
    p.y = y;
    p.dt = y_dt;
    p.y_stride = y_stride;
    if (coded) {
        if ((st = need(x, "x", 16)) != EXL3_OK) return st;
        if (x_stride % 16)
            return set_error(EXL3_ERR_INVALID_ARG, "x: row stride %lld is not a multiple of 16", (long long)x_stride);
        if ((st = need(x_scale, "x_scale", 4)) != EXL3_OK) return st;
        if (xs_t < 0 || xs_b < 0 || xs_t > (1ll << 32) || xs_b > (1ll << 32))
            return set_error(EXL3_ERR_INVALID_ARG, "x_scale: strides %lld and %lld are not in [0, 2^32]", (long long)xs_t, (long long)xs_b);
        const size_t s_bytes = (size_t)((T - 1) * xs_t + (blocks_of(n_in) - 1) * xs_b + 1) * 4;
        if ((st = check_apart(yr, "y", x_scale, s_bytes, "x_scale")) != EXL3_OK) return st;
        p.x = reinterpret_cast<const uint8_t *>(x);
        p.x_stride = x_stride;
        p.xs = x_scale;
        p.xs_t = xs_t;
        p.xs_b = xs_b;
        return launch_linear8(p, (cudaStream_t)stream);
    }
    const Linear8Ws m(ws, T, n_in);
    if ((st = check_ws(ws, ws_bytes, m.bytes)) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", ws, m.bytes, "the workspace")) != EXL3_OK) return st;
    if ((st = launch_quantize8({x, x_dt, T, n_in, x_stride, 1, m.codes, m.scale}, (cudaStream_t)stream)) != EXL3_OK) return st;
    p.x = m.codes;
    p.x_stride = n_in;
    p.xs = m.scale;
    p.xs_t = 1;
    p.xs_b = T;
    p.behind = true;
    return launch_linear8(p, (cudaStream_t)stream);
}

size_t exl3_expert_layer_workspace_bytes(int64_t T, int64_t hidden, int64_t inner, int n_experts, int top_k) {
    if (!layer_ok(T, hidden, inner, n_experts, top_k))
        return 0;
    ExpertLaunch p = {};
    p.T = T;
    p.H = (int)hidden;
    p.F = (int)inner;
    p.E = n_experts;
    p.top_k = top_k;
    return carve_layer(p, nullptr);
}

exl3_status exl3_expert_layer(const void *x, int dt, int64_t T, int64_t x_stride, const void *router, int r_dt,
                              const int32_t *ids, const float *weights, int top_k, int normalize, int n_experts,
                              const exl3_coded *experts, int64_t hidden, int64_t inner, int K, int K_down, int transposed,
                              void *y, int64_t y_stride, void *ws, size_t ws_bytes, void *stream) {
    exl3_status st;
    if ((st = check_16bit(dt)) != EXL3_OK) return st;
    if (n_experts < 1 || n_experts > kMaxExperts)
        return set_error(EXL3_ERR_UNSUPPORTED, "%d experts: 1 to %d are supported", n_experts, kMaxExperts);
    if (top_k < 1 || top_k > kMaxPicks || top_k > n_experts)
        return set_error(EXL3_ERR_UNSUPPORTED, "%d picks of %d experts: 1 to %d are supported, no more than experts", top_k, n_experts, kMaxPicks);
    if (T < 0 || T > kMaxLayerTokens || T * top_k > kMaxPairs)
        return set_error(EXL3_ERR_UNSUPPORTED, "%lld tokens of %d picks: up to %lld tokens and %lld pairs are supported (exl3_expert_linear takes more)",
                         (long long)T, top_k, (long long)kMaxLayerTokens, (long long)kMaxPairs);
    if (!layer_side(hidden) || !layer_side(inner))
        return set_error(EXL3_ERR_UNSUPPORTED, "hidden and inner must be multiples of 128 up to %lld, got %lld and %lld",
                         (long long)kMaxLayerSide, (long long)hidden, (long long)inner);
    if (!exl3_supports_k(K) || !exl3_supports_k(K_down))
        return set_error(EXL3_ERR_UNSUPPORTED, "K=%d, K_down=%d is not supported", K, K_down);
    if (!experts)
        return set_error(EXL3_ERR_INVALID_ARG, "experts is NULL");
    static const char *const names[3][4] = {{"gate codes", "gate su", "gate sv", "gate scale"},
                                            {"up codes", "up su", "up sv", "up scale"},
                                            {"down codes", "down su", "down sv", "down scale"}};
    for (int m = 0; m < 3; m++) {
        if ((st = need(experts[m].codes, names[m][0], 16)) != EXL3_OK) return st;
        if ((st = need(experts[m].su, names[m][1], 16)) != EXL3_OK) return st;
        if ((st = need(experts[m].sv, names[m][2], 16)) != EXL3_OK) return st;
        if ((st = need(experts[m].scale, names[m][3], 4)) != EXL3_OK) return st;
    }
    if (router) {
        if (r_dt != dt && r_dt != EXL3_F32)
            return set_error(EXL3_ERR_INVALID_ARG, "router's dtype %d is neither x's nor EXL3_F32", r_dt);
        if (!aligned(router, r_dt == EXL3_F32 ? 4 : 2))
            return set_error(EXL3_ERR_INVALID_ARG, "router is not aligned");
        if (ids || weights)
            return set_error(EXL3_ERR_INVALID_ARG, "ids and weights do not go with a router");
    } else if (T) {
        if ((st = need(ids, "ids", 4)) != EXL3_OK) return st;
        if ((st = need(weights, "weights", 4)) != EXL3_OK) return st;
    }
    const Rows xr{x, T, hidden, x_stride}, yr{y, T, hidden, y_stride};
    if ((st = check_rows(xr, "x")) != EXL3_OK) return st;
    if ((st = check_rows(yr, "y")) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", xr, "x")) != EXL3_OK) return st;
    for (int m = 0; m < 3; m++) {
        const size_t n = (size_t)n_experts * 4, left = n * (m == 2 ? inner : hidden), right = n * (m == 2 ? hidden : inner);
        const size_t bytes = (size_t)n_experts * hidden * inner * (m == 2 ? K_down : K) / 8;
        if ((st = check_apart(yr, "y", experts[m].codes, bytes, names[m][0])) != EXL3_OK) return st;
        if ((st = check_apart(yr, "y", experts[m].su, transposed ? right : left, names[m][1])) != EXL3_OK) return st;
        if ((st = check_apart(yr, "y", experts[m].sv, transposed ? left : right, names[m][2])) != EXL3_OK) return st;
        if ((st = check_apart(yr, "y", experts[m].scale, n, names[m][3])) != EXL3_OK) return st;
    }
    const size_t picks = (size_t)(T * top_k) * 4;
    if ((st = check_apart(yr, "y", router, (size_t)n_experts * hidden * (r_dt == EXL3_F32 ? 4 : 2), "router")) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", ids, picks, "ids")) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", weights, picks, "weights")) != EXL3_OK) return st;
    if (T == 0)
        return EXL3_OK;
    ExpertLaunch p = {};
    p.x = x;
    p.dt = dt;
    p.T = T;
    p.x_stride = x_stride;
    p.H = (int)hidden;
    p.F = (int)inner;
    p.E = n_experts;
    p.top_k = top_k;
    p.router = router;
    p.r_dt = r_dt;
    p.normalize = normalize != 0;
    ExpertMatrix *const to[3] = {&p.gate, &p.up, &p.down};
    for (int m = 0; m < 3; m++) {
        const exl3_coded &c = experts[m];
        *to[m] = {reinterpret_cast<const uint32_t *>(c.codes), transposed ? c.sv : c.su, transposed ? c.su : c.sv, c.scale};
    }
    p.K = K;
    p.K_down = K_down;
    p.transposed = transposed ? 1 : 0;
    p.y = y;
    p.y_stride = y_stride;
    p.ids = const_cast<int32_t *>(ids);            // (written only with a router)
    p.weights = const_cast<float *>(weights);
    const size_t want = carve_layer(p, ws);
    if ((st = check_ws(ws, ws_bytes, want)) != EXL3_OK) return st;
    if ((st = check_apart(yr, "y", ws, want, "the workspace")) != EXL3_OK) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if ((st = launch_expert_route(p, s)) != EXL3_OK) return st;
    if ((st = launch_expert_up(p, s)) != EXL3_OK) return st;
    return launch_expert_down(p, s);
}

}  // extern "C"
