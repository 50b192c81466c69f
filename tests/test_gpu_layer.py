"""Norms, blocks in 8 bits and products with them on the GPU, against their formulas
in 64 bits.

Tolerances.  A rounding to a type is off by at most half a step: u = 2^-8 (bfloat16),
2^-11 (float16) of the value, half a subnormal step below (2^-25 for float16); e4m3 by
2^-4 of the value or 2^-10 under 2^-6, before the block's scale.

Norm: a row's sum of squares is a chain of at most 8 * 4 fused additions a thread, five
across a warp and five across warps, all terms positive: 42 * 2^-24 of it; half of that
reaches s, whose own steps (mean, eps, root, two products) add 6 * 2^-24: 32 * 2^-24 in all.

Its gradient: sum(g h) is off by 44 * 2^-24 of sum |g h|, s^3 by 100 * 2^-24, each
operation by 2^-24 more: 160 * 2^-24 of |s g| + |h| s^3 mean|g h| + |dh|.  dweight adds
terms that are each off by 40 * 2^-24, in chains of at most 2 * T / 152 + 10 + T / 32.

Product in 8 bits: the codes' products are exact in binary32's 24 bits; a tensor-core
step adds 32 of them to an accumulator and may cut below 2^-20 of the largest, four
steps to a block, and the blocks are added in binary32 under their scales (four roundings
and at most 8 sums of parts): 2^-17 of the sum of magnitudes covers up to 40 blocks.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
F = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.fail("CUDA is required for -m gpu tests")
    import __graft_entry__
    __graft_entry__.build()
    import exl3_trellis_weight_gb300 as ex
    return ex


@pytest.fixture(autouse=True)
def _no_expired_waits(ex):
    yield
    assert ex.wait_timeouts() == 0


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def acts(g, T, n, dt, wide=False, scale=1.0):
    x = torch.randn(T, n, generator=g, device=DEV) * torch.exp(torch.randn(T, 1, generator=g, device=DEV)) * scale
    if n > 3:
        x[:, 3] *= 15.0
    if not wide:
        return x.to(DT[dt])
    buf = torch.full((T, n + 37), 7.0, dtype=DT[dt], device=DEV)
    buf[:, 5:5 + n] = x.to(DT[dt])
    return buf[:, 5:5 + n]


def within(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


def spread(scale, T, n, rows=1):
    return scale.double().repeat_interleave(rows, 0)[:T].repeat_interleave(128, 1)[:, :n]


def norm64(h, w, eps):
    s = 1.0 / torch.sqrt(h.double().pow(2).mean(1, keepdim=True) + eps)
    return h.double() * s * w.double(), s


def check_blocks(codes, scale, v, off, rows=1):
    """codes and scales stand for v, known up to a relative error `off`."""
    T, n = v.shape
    nb = -(-n // 128)
    pad = torch.nn.functional.pad(v.abs(), (0, 128 * nb - n, 0, -T % rows)).view(-1, rows, nb, 128)
    m = pad.amax((1, 3)).clamp_min(2.0 ** -96)
    within(scale, m / 448.0, (off + F) * m / 448.0)
    s = spread(scale, T, n, rows)
    # the factor 448 / m and the product with it, two roundings, before e4m3's
    within(codes.double() * s, v, torch.maximum(v.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -4) * (1 + 20 * F) + 2 * (off + 4 * F) * v.abs())


SHAPES = [(1, 1), (1, 64), (3, 127), (2, 128), (5, 129), (1, 4096), (7, 1001), (400, 256), (333, 1000), (310, 2048), (700, 4097),
          (2, 8192), (3, 8200), (400, 5000), (5, 20001), (2, 32768), (306, 16384)]


@pytest.mark.parametrize("T,n", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("residual,wide,w32", [(False, False, False), (True, True, True), (True, False, False), (False, True, False)])
def test_norm(ex, T, n, dt, residual, wide, w32):
    g = gen(T + n)
    x = acts(g, T, n, dt, wide)
    r = acts(g, T, n, dt, wide) if residual else None
    w = (1.0 + 0.3 * torch.randn(n, generator=g, device=DEV)).to(torch.float32 if w32 else DT[dt])
    eps = 1e-5
    got = ex.rms_norm(x, w, eps, residual=r, want_y=True, want_y8=True)
    h = x
    if residual:
        h = (x.float() + r.float()).to(DT[dt])
        assert torch.equal(got["h"], h)
    else:
        assert got["h"] is None
    y, _ = norm64(h, w, eps)
    within(got["y"], y, (U[dt] * (1 + 64 * F) + 32 * F) * y.abs() + TINY[dt])
    check_blocks(got["y8"], got["scale"], y, 32 * F)
    assert got["y8"].dtype is E4M3 and got["scale"].shape == (T, -(-n // 128))
    # one output at a time is the same
    assert torch.equal(ex.rms_norm(x, w, eps, residual=r)["y"], got["y"])
    q = ex.rms_norm(x, w, eps, residual=r, want_y=False, want_y8=True)
    assert q["y"] is None and torch.equal(q["y8"].view(torch.uint8), got["y8"].view(torch.uint8)) and torch.equal(q["scale"], got["scale"])


def test_norm_in_place_and_into_columns(ex):
    g = gen(3)
    T, n = 350, 768
    x, r, w = acts(g, T, n, "bf16"), acts(g, T, n, "bf16"), torch.rand(n, generator=g, device=DEV)
    want = ex.rms_norm(x, w, residual=r)
    # the residual stream updated where it lies, the result over x
    x1, r1 = x.clone(), r.clone()
    got = ex.rms_norm(x1, w, residual=r1, h=r1, out=x1)
    assert got["h"] is r1 and got["y"] is x1
    assert torch.equal(r1, want["h"]) and torch.equal(x1, want["y"])
    # into columns of a wider buffer, whose others stay
    buf = torch.full((T, n + 100), 3.0, dtype=torch.bfloat16, device=DEV)
    ex.rms_norm(x, w, residual=r, out=buf[:, 50:50 + n])
    # (the order of a row's sum goes by alignment)
    y, _ = norm64(want["h"], w, 1e-6)
    within(buf[:, 50:50 + n], y, (U["bf16"] * (1 + 64 * F) + 32 * F) * y.abs())
    assert bool((buf[:, :50] == 3).all()) and bool((buf[:, 50 + n:] == 3).all())


def test_norm_of_zeros_large_and_small_rows(ex):
    n = 512
    x = torch.zeros(5, n, dtype=torch.bfloat16, device=DEV)
    x[1] = 1e-30
    x[2] = 1e18
    x[3, 7] = 1e-3
    w = torch.ones(n, device=DEV)
    got = ex.rms_norm(x, w, 1e-6, want_y8=True)
    y, _ = norm64(x, w, 1e-6)
    within(got["y"], y, (U["bf16"] + 40 * F) * y.abs())
    check_blocks(got["y8"], got["scale"], y, 32 * F)
    assert bool((got["y"][0] == 0).all()) and bool((got["y8"][0].float() == 0).all())


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_rows_that_are_not_numbers_stay_alone(ex, value):
    g = gen(5)
    T, n = 330, 640
    x, w = acts(g, T, n, "bf16"), torch.rand(n, generator=g, device=DEV)
    bad = x.clone()
    bad[17, 200] = value
    a, b = ex.rms_norm(x, w, want_y8=True), ex.rms_norm(bad, w, want_y8=True)
    keep = torch.arange(T, device=DEV) != 17
    for k in ("y", "scale"):
        assert torch.equal(a[k][keep], b[k][keep])
    assert torch.equal(a["y8"].view(torch.uint8)[keep], b["y8"].view(torch.uint8)[keep])
    assert not bool(b["y"][17].float().isfinite().all())
    # blocks of a matrix: the block alone, as a whole
    c0, s0 = ex.quantize8(x)
    c1, s1 = ex.quantize8(bad)
    v0, v1 = c0.float() * spread(s0, T, n).float(), c1.float() * spread(s1, T, n).float()
    assert bool(v1[17, 128:256].isnan().all())
    v1[17, 128:256] = v0[17, 128:256]
    assert torch.equal(v0, v1)


@pytest.mark.parametrize("T,n", SHAPES + [(1300, 512), (4000, 64)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("with_dh,wide,w32", [(False, False, False), (True, True, True)])
def test_norm_gradient(ex, T, n, dt, with_dh, wide, w32):
    g = gen(T * 3 + n)
    h, dy = acts(g, T, n, dt, wide), acts(g, T, n, dt, wide, 0.1)
    dh = acts(g, T, n, dt, wide, 0.1) if with_dh else None
    w = (1.0 + 0.3 * torch.randn(n, generator=g, device=DEV)).to(torch.float32 if w32 else DT[dt])
    eps = 1e-5
    got = ex.rms_norm_backward(dy, h, w, eps, dh=dh)
    h64, g64 = h.double(), dy.double() * w.double()
    _, s = norm64(h, w, eps)
    dx = s * g64 - h64 * s.pow(3) * (g64 * h64).mean(1, keepdim=True)
    size = (s * g64).abs() + h64.abs() * s.pow(3) * (g64 * h64).abs().mean(1, keepdim=True)
    if with_dh:
        dx, size = dx + dh.double(), size + dh.double().abs()
    within(got["dx"], dx, U[dt] * dx.abs() + 161 * F * size + TINY[dt])
    terms = dy.double() * h64 * s
    dw, udt = terms.sum(0), "fp32" if w32 else dt
    within(got["dweight"], dw, U[udt] * dw.abs() + (60 + T / 16) * F * terms.abs().sum(0) + TINY[udt])
    alone = ex.rms_norm_backward(dy, h, w, eps, dh=dh, want_dweight=False)
    assert alone["dweight"] is None and torch.equal(alone["dx"], got["dx"])
    if T > 1:      # the same again, and in place
        again = ex.rms_norm_backward(dy, h, w, eps, dh=dh)
        assert torch.equal(again["dweight"], got["dweight"])
        over = dy.clone() if not with_dh else dh.clone()
        r = ex.rms_norm_backward(over if not with_dh else dy, h, w, eps, dh=over if with_dh else None, dx=over)
        if not wide:
            assert torch.equal(over, got["dx"]) and torch.equal(r["dweight"], got["dweight"])


@pytest.mark.parametrize("n", [300, 1001, 2048, 9000, 20000])
def test_norm_gradient_of_large_rows(ex, n):
    """Sums of squares and of products beyond binary32's range, one of them and both, among
    ordinary rows: each row as exact as another."""
    g = gen(n)
    T = 9
    h, dy = torch.randn(T, n, generator=g, device=DEV), torch.randn(T, n, generator=g, device=DEV)
    h *= torch.tensor([1, 1e19, 1, 1e19, 1e-3, 1e30, 1e25, 1, 3e37], device=DEV)[:, None]
    dy *= torch.tensor([1, 1, 1e36, 1e30, 1, 1e-10, 1e25, 1e20, 1], device=DEV)[:, None]
    h, dy = h.bfloat16(), dy.bfloat16()
    w = 0.5 + torch.rand(n, generator=g, device=DEV)
    got = ex.rms_norm_backward(dy, h, w, 1e-6)
    h64, g64 = h.double(), dy.double() * w.double()
    _, s = norm64(h, w, 1e-6)
    m = (g64 * h64).mean(1, keepdim=True)
    dx = s * g64 - h64 * s.pow(3) * m
    size = (s * g64).abs() + h64.abs() * s.pow(3) * (g64 * h64).abs().mean(1, keepdim=True)
    within(got["dx"], dx, U["bf16"] * dx.abs() + 161 * F * size + 2.0 ** -133)
    terms = dy.double() * h64 * s
    within(got["dweight"], terms.sum(0), (61 + T / 16) * F * terms.abs().sum(0))


def test_norm_gradient_against_differences(ex):
    """Along a direction: (f(h + d) - f(h - d)) / 2 in 64 bits of f = sum(dy . y); with d = 1e-4 of
    a unit row its own error is below 1e-7 of f's third derivatives, of the order of |dy| / rms^3."""
    g = gen(11)
    T, n, eps = 9, 333, 1e-6
    h, dy = (torch.randn(T, n, generator=g, device=DEV).half() for _ in range(2))
    w = torch.rand(n, generator=g, device=DEV) + 0.5
    d, e = torch.randn(T, n, generator=g, device=DEV).double(), torch.randn(n, generator=g, device=DEV).double()
    got = ex.rms_norm_backward(dy, h, w, eps)

    def f(t):
        hh, ww = h.double() + t * d, w.double() + t * e
        return float((dy.double() * hh / torch.sqrt(hh.pow(2).mean(1, keepdim=True) + eps) * ww).sum())

    num = (f(1e-4) - f(-1e-4)) / 2e-4
    ana = float((got["dx"].double() * d).sum() + (got["dweight"].double() * e).sum())
    # dx is rounded to float16: independent errors of at most 2^-11 of each
    tol = 6 * 2.0 ** -11 / math.sqrt(3) * float((got["dx"].double() * d).norm()) + 1e-5 * abs(num)
    assert abs(num - ana) <= tol, (num, ana, tol)


def test_norm_gradient_flows_through_the_calls(ex):
    g = gen(12)
    T, n = 65, 384
    x, r = acts(g, T, n, "fp16"), acts(g, T, n, "fp16")
    w = torch.rand(n, generator=g, device=DEV) + 0.5
    dy, dh = acts(g, T, n, "fp16", scale=0.1), acts(g, T, n, "fp16", scale=0.1)
    h = (x.float() + r.float()).half()
    want = ex.rms_norm_backward(dy, h, w, dh=dh)
    xs, rs, ws = (t.clone().requires_grad_() for t in (x, r, w))
    o = ex.rms_norm(xs, ws, residual=rs)
    torch.autograd.backward([o["y"], o["h"]], [dy, dh])
    assert torch.equal(xs.grad, want["dx"]) and torch.equal(rs.grad, want["dx"]) and torch.equal(ws.grad, want["dweight"])
    # y alone, h alone, no residual, a frozen weight, an expanded gradient
    xs = x.clone().requires_grad_()
    ex.rms_norm(xs, w, residual=r)["y"].backward(dy)
    assert torch.equal(xs.grad, ex.rms_norm_backward(dy, h, w)["dx"])
    xs = x.clone().requires_grad_()
    ex.rms_norm(xs, w, residual=r)["h"].backward(dh)
    assert torch.equal(xs.grad, dh)
    xs = x.clone().requires_grad_()
    ex.rms_norm(xs, w)["y"].backward(dy[:1].expand(T, n))
    assert torch.equal(xs.grad, ex.rms_norm_backward(dy[:1].expand(T, n).contiguous(), x, w)["dx"])
    with pytest.raises(ValueError, match="gradient"):
        ex.rms_norm(xs, w, want_y8=True)
    with torch.no_grad():
        ex.rms_norm(xs, w, want_y8=True)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,n,wide", [(1, 1, False), (1, 128, False), (127, 129, True), (128, 128, False), (129, 256, True), (300, 1000, False),
                                      (5, 65536, False), (2049, 384, False), (700, 333, False)])
def test_blocks_bit_for_bit(ex, block, dt, T, n, wide):
    """The definition in binary32 on the CPU, whose divisions are IEEE's."""
    x = acts(gen(T + n), T, n, dt, wide)
    if T > 100:
        x[50] = 0
    codes, scale = ex.quantize8(x, block_rows=block)
    v = x.float().cpu()
    R, N = -(-T // block), -(-n // 128)
    b = torch.nn.functional.pad(v, (0, 128 * N - n, 0, block * R - T)).view(R, block, N, 128)
    m = b.abs().amax((1, 3)).clamp_min(2.0 ** -96)
    inv = torch.full_like(m, 448.0) / m
    q = (b * inv[:, None, :, None]).clamp(-448, 448).view(R * block, N * 128)[:T, :n].to(E4M3)
    assert torch.equal(scale.cpu(), m / torch.full_like(m, 448.0))
    assert torch.equal(codes.cpu().view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("T,n", [(1, 2), (3, 130), (340, 1002), (5, 4100), (700, 2050), (310, 9010), (2, 20006)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_even_sizes(ex, T, n, dt):
    """Rows of whole pairs that are no multiples of 16 bytes; the same from and into columns at even and
    odd places of a wider buffer."""
    test_norm(ex, T, n, dt, True, False, True)
    test_norm(ex, T, n, dt, False, False, False)
    test_norm_gradient(ex, T, n, dt, True, False, True)
    test_norm_gradient(ex, T, n, dt, False, False, False)
    for block in (1, 128):
        test_blocks_bit_for_bit(ex, block, dt, T, n, False)
    test_blocks_bit_for_bit(ex, 1, "fp32", T, n, False)
    g = gen(n)
    x, w = acts(g, T, n, dt), torch.rand(n, generator=g, device=DEV).to(DT[dt])
    y, _ = norm64(x, w, 1e-6)
    for at in (0, 1, 2, 8):
        buf, out = (torch.full((T, n + 12), 3.0, dtype=DT[dt], device=DEV) for _ in range(2))
        buf[:, at:at + n] = x
        got = ex.rms_norm(buf[:, at:at + n], w, 1e-6, out=out[:, at:at + n], want_y8=True)
        within(out[:, at:at + n], y, (U[dt] * (1 + 64 * F) + 32 * F) * y.abs() + TINY[dt])
        assert bool((out[:, :at] == 3).all()) and bool((out[:, at + n:] == 3).all())
        check_blocks(got["y8"], got["scale"], y, 32 * F)


def weights8(g, rows, cols):
    w = (torch.randn(rows, cols, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)
    return w, 0.001 * torch.exp(torch.randn(-(-rows // 128), -(-cols // 128), generator=g, device=DEV))


def product64(codes, scale, w, w_scale, tr):
    T, n = codes.shape
    x = codes.double() * spread(scale, T, n)
    W = w.double() * spread(w_scale, *w.shape, 128)
    W = W.t() if tr else W
    return x @ W, x.abs() @ W.abs()


TOKENS = [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 300, 513]


@pytest.mark.parametrize("rows,cols", [(16, 16), (128, 128), (144, 1280), (1040, 272), (2000, 1008), (256, 4096)])
@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_product(ex, rows, cols, tr, dt):
    g = gen(rows + cols + tr)
    w, ws = weights8(g, rows, cols)
    n_in = cols if tr else rows
    for T in TOKENS:
        codes, scale = ex.quantize8(acts(g, T, n_in, dt))
        y = ex.linear8(codes, w, ws, scale, transposed=tr, dtype=DT[dt])
        ref, size = product64(codes, scale, w, ws, tr)
        within(y, ref, U[dt] * ref.abs() + 2.0 ** -17 * size + TINY[dt])
        # scales by token, as a contiguous tensor: the same
        assert torch.equal(y, ex.linear8(codes, w, ws, scale.contiguous(), transposed=tr, dtype=DT[dt]))


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("T", [1, 20, 64, 70, 1500, 5000])
def test_product_of_16_bits(ex, tr, T):
    """x in 16 bits is the product of its blocks; rows of a wider buffer, results into one."""
    g = gen(T)
    rows, cols = (1280, 512) if tr else (512, 1280)
    w, ws = weights8(g, rows, cols)
    x = acts(g, T, 512, "bf16", wide=True)
    want = ex.linear8(*(lambda c, s: (c, w, ws, s))(*ex.quantize8(x)), transposed=tr)
    assert torch.equal(ex.linear8(x, w, ws, transposed=tr), want)
    buf = torch.full((T, 1280 + 64), 3.0, dtype=torch.bfloat16, device=DEV)
    ex.linear8(x, w, ws, transposed=tr, out=buf[:, 33:33 + 1280])
    assert torch.equal(buf[:, 33:33 + 1280], want) and bool((buf[:, :33] == 3).all()) and bool((buf[:, 33 + 1280:] == 3).all())
    ref, size = product64(*ex.quantize8(x), w, ws, tr)
    within(want, ref, U["bf16"] * ref.abs() + 2.0 ** -17 * size)


@pytest.mark.parametrize("T,rows,cols,tr", [(40, 16384, 256, False), (200, 256, 16384, True), (3, 65536, 128, False), (130, 128, 65536, True)])
def test_product_of_many_inputs(ex, T, rows, cols, tr):
    g = gen(T)
    w, ws = weights8(g, rows, cols)
    codes, scale = ex.quantize8(acts(g, T, max(rows, cols), "fp16"))
    y = ex.linear8(codes, w, ws, scale, transposed=tr, dtype=torch.float16)
    ref, size = product64(codes, scale, w, ws, tr)
    within(y, ref, U["fp16"] * ref.abs() + 2.0 ** -17 * max(rows, cols) / 5120 * size + TINY["fp16"])


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("tr", [False, True])
def test_product_keeps_tokens_apart(ex, T, tr):
    """A token that is no number, and one whose scale is none, give none; the others are as before."""
    g = gen(8)
    w, ws = weights8(g, 384, 384)
    codes, scale = ex.quantize8(acts(g, T, 384, "bf16"))
    y0 = ex.linear8(codes, w, ws, scale, transposed=tr)
    bad = codes.clone()
    bad.view(torch.uint8)[2, 130] = 0x7F
    bs = scale.clone()
    bs[4, 1] = math.inf
    y1 = ex.linear8(bad, w, ws, bs, transposed=tr)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[2] = keep[4] = False
    assert torch.equal(y0[keep], y1[keep])
    assert not bool(y1[2].float().isfinite().any()) and not bool(y1[4].float().isfinite().any())


def test_product_gradient(ex):
    """x's gradient is the product with the other transposition; with x and dy whose blocks are
    exact in e4m3 the calls are linear, and differences give the same."""
    g = gen(9)
    T, rows, cols = 50, 256, 384
    w, ws = weights8(g, rows, cols)

    def exact(T, n):       # values that are codes under a power-of-two scale, 448 among each block's
        v = torch.randint(-8, 9, (T, n), generator=g, device=DEV).float()
        v[:, ::128] = 448.0
        return v.to(torch.bfloat16)

    x, dy, d = exact(T, rows), exact(T, cols), exact(T, rows)
    xr = x.clone().requires_grad_()
    y = ex.linear8(xr, w, ws)
    y.backward(dy)
    assert torch.equal(xr.grad, ex.linear8(dy, w, ws, transposed=True))
    W = w.double() * spread(ws, rows, cols, 128)
    ref = dy.double() @ W.t()
    within(xr.grad, ref, U["bf16"] * ref.abs() + 2.0 ** -17 * (dy.double().abs() @ W.abs().t()))
    num = float((dy.double() * (d.double() @ W)).sum())         # f(x + d) - f(x) of the linear f
    ana = float((xr.grad.double() * d.double()).sum())
    assert abs(num - ana) <= 6 * U["bf16"] / math.sqrt(3) * float((xr.grad.double() * d.double()).norm()) + 1e-4 * abs(num)
    with pytest.raises(ValueError, match="gradient"):
        ex.linear8(xr, w, ws.clone().requires_grad_())


def test_in_a_graph_on_another_stream_and_without_tokens(ex):
    g = gen(10)
    T, n = 40, 512
    w8, ws = weights8(g, n, 768)
    x, r, w = acts(g, T, n, "bf16"), acts(g, T, n, "bf16"), torch.rand(n, generator=g, device=DEV)

    def chain():
        o = ex.rms_norm(x, w, residual=r, want_y=False, want_y8=True)
        return ex.linear8(o["y8"], w8, ws, o["scale"]), ex.linear8(o["h"], w8, ws)

    want = chain()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = chain()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    x.copy_(acts(g, T, n, "bf16"))
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(chain(), got))
    e = x[:0]
    assert ex.rms_norm(e, w, residual=e, want_y8=True)["y8"].shape == (0, n)
    assert ex.linear8(e, w8, ws).shape == (0, 768) and ex.quantize8(e, 128)[1].shape == (0, 4)
    assert ex.linear8(e.to(E4M3), w8, ws, torch.empty(0, 4, device=DEV)).shape == (0, 768)
    b = ex.rms_norm_backward(e, e, w)
    assert b["dx"].shape == (0, n) and bool((b["dweight"] == 0).all())


def test_threads_that_call_at_once(ex):
    """Six host threads, each with its stream and sizes: the same results as alone."""
    import threading
    g = gen(21)
    x = [acts(g, 64 + 100 * i, 512 + 128 * i, "bf16") for i in range(6)]
    w = [torch.rand(512 + 128 * i, generator=g, device=DEV) for i in range(6)]
    m = [ex.quantize8(torch.randn(512 + 128 * i, 640, generator=g, device=DEV), block_rows=128) for i in range(6)]

    def work(i):
        n = ex.rms_norm(x[i], w[i], want_y8=True)
        b = ex.rms_norm_backward(x[i], x[i], w[i])
        return n["y"], b["dx"], b["dweight"], ex.linear8(n["y8"], *m[i], n["scale"]), ex.linear8(x[i], *m[i])

    want = [work(i) for i in range(6)]
    torch.cuda.synchronize()
    other = []

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = work(i)
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    other.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not other


def test_a_captured_backward_pass(ex):
    """Norm and 8-bit product with their gradients in a graph, replayed with other inputs."""
    g = gen(22)
    m = ex.quantize8(torch.randn(640, 256, generator=g, device=DEV), block_rows=128)
    x, w = acts(g, 40, 640, "bf16").requires_grad_(), torch.rand(640, generator=g, device=DEV).requires_grad_()

    def step():
        y = ex.linear8(ex.rms_norm(x, w)["y"], *m)
        return torch.autograd.grad(y, [x, w], torch.ones_like(y))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        x.copy_(acts(g, 40, 640, "bf16"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_offsets_beyond_32_bits(ex):
    """2.3e9 values: the first row, the last and the one across 2^31 are as exact as any."""
    g = gen(23)
    T, n = 140000, 16384
    x = torch.empty(T, n, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    w = torch.rand(n, generator=g, device=DEV)
    m, ms = ex.quantize8(torch.randn(64, n, generator=g, device=DEV), block_rows=128)
    at = [0, 2 ** 31 // n - 1, 2 ** 31 // n, T - 1]
    r = ex.rms_norm(x, w, 1e-6, want_y8=True)
    y, s = norm64(x[at], w, 1e-6)
    within(r["y"][at], y, (U["bf16"] * (1 + 64 * F) + 32 * F) * y.abs())
    check_blocks(r["y8"][at], r["scale"][at], y, 32 * F)
    p = ex.linear8(r["y8"], m, ms, r["scale"], transposed=True)
    ref, size = product64(r["y8"][at], r["scale"][at], m, ms, True)
    within(p[at], ref, U["bf16"] * ref.abs() + 2.0 ** -17 * n / 5120 * size)
    dy = r["y"]
    del r, p
    got = ex.rms_norm_backward(dy, x, w, 1e-6, want_dweight=False)["dx"]
    h64, g64 = x[at].double(), dy[at].double() * w.double()
    dx = s * g64 - h64 * s.pow(3) * (g64 * h64).mean(1, keepdim=True)
    size = (s * g64).abs() + h64.abs() * s.pow(3) * (g64 * h64).abs().mean(1, keepdim=True)
    within(got[at], dx, U["bf16"] * dx.abs() + 161 * F * size)
    del got, dy
    codes, scale = ex.quantize8(x, block_rows=128)
    first = (T - 1) // 128 * 128
    check_blocks(codes[first:], scale[first // 128:], x[first:].double(), 0.0, rows=128)
