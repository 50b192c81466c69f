"""Whole expert layers on the GPU, against the definition in 64 bits.

Tolerances.  A pair of a token and an expert adds P = w (h D) with h = silu(a) b, a = x G,
b = x U.  The rotated x and the rotated inner activations are rounded to binary16: r, the
standard deviation of an element's relative error, is 2^-11 / sqrt(3) at most for x in
bfloat16.  For float16 both are kept in two parts, 22 bits, and what is left are the sums in
binary32 of up to some thousand products, 2^-20 of their root mean square.  Rotations keep
norms, so in every channel
  a and b are off by r times the root mean square of a / right (b / right) times |right|,
  h by 1.1 |b| da + |silu(a)| db (|silu'| is 1.1 at most), a share q of h . left in norm,
  P by (r + q) times the root mean square of P / right, times |right|:
codes that are random prefer no direction.  Six of these, added up over a token's pairs as
they are, cover what chance gives.  Weights come from logits and a softmax in binary32:
2^-16 of |P|.  One rounding of the result, 2^-8 or 2^-11 of itself (2^-25 where float16 is
subnormal), comes on top.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_linear import DEV, DT, U, acts, coded, gen, weight64  # noqa: E402


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


class Experts:
    """Coded experts and their matrices in 64 bits, G and U [H, F], D [F, H]."""

    def __init__(self, g, E, H, F, K, Kd, tr):
        self.E, self.H, self.F, self.K, self.Kd, self.tr = E, H, F, K, Kd, tr
        up, down = ((F, H), (H, F)) if tr else ((H, F), (F, H))
        self.gate, self.up, self.down = coded(g, *up, K, (E,)), coded(g, *up, K, (E,)), coded(g, *down, Kd, (E,))
        for m in (self.gate, self.up):                    # a and b of the order of one
            m[3].mul_(1.5 / math.sqrt(H))
        self._dense = {}

    def dense(self, e):
        if e not in self._dense:
            ms = [weight64(*(t[e] for t in m[:3]), K, m[3][e]) for m, K in ((self.gate, self.K), (self.up, self.K), (self.down, self.Kd))]
            self._dense[e] = [m.t() if self.tr else m for m in ms]
        return self._dense[e]

    def right(self, m, e):
        return (m[1] if self.tr else m[2])[e].double()

    def left(self, m, e):
        return (m[2] if self.tr else m[1])[e].double()

    def run(self, ex, x, top_k, **kw):
        return ex.expert_layer(x, self.gate, self.up, self.down, self.K, top_k, transposed=self.tr, K_down=self.Kd, **kw)


def rms(v, right):
    live = right != 0
    return (v[:, live] / right[live]).pow(2).mean(1, keepdim=True).sqrt() * right.abs()


def expected(m, x, ids, weights, dt):
    """(y, tolerance) in 64 bits for these picks."""
    y = torch.zeros(x.shape[0], m.H, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(y)
    r = 2.0 ** -11 / math.sqrt(3) if dt == "bf16" else 2.0 ** -20
    for e in range(m.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        G, Up, D = m.dense(e)
        xe, w = x[t].double(), weights[t, j].double()[:, None]
        a, b = xe @ G, xe @ Up
        s = a * torch.sigmoid(a)
        dh = 1.1 * b.abs() * r * rms(a, m.right(m.gate, e)) + s.abs() * r * rms(b, m.right(m.up, e))
        left = m.left(m.down, e)
        q = (dh * left).norm(dim=1, keepdim=True) / (s * b * left).norm(dim=1, keepdim=True).clamp_min(1e-300)
        P = w * (s * b @ D)
        y.index_add_(0, t, P)
        tol.index_add_(0, t, 6 * (r + q) * rms(P, m.right(m.down, e)) + 2.0 ** -16 * P.abs())
    return y, tol + U[dt] * y.abs() * (1 + 2.0 ** -10) + 2.0 ** -25


def within(got, want):
    y, tol = want
    bad = ~((got.double() - y).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - y).abs() / tol).max()))


def picks(x, router, top_k, normalize=True):
    p = torch.softmax(x.double() @ router.double().t(), 1)
    w, ids = torch.sort(p, dim=1, descending=True, stable=True)
    w, ids = w[:, :top_k], ids[:, :top_k]
    return ids, w / w.sum(1, keepdim=True) if normalize else w


def a_router(g, E, H, dt):
    return (torch.randn(E, H, generator=g, device=DEV) / math.sqrt(H)).to(dt)


SHAPES = [(1, 128, 128, 1), (5, 256, 384, 5), (8, 640, 256, 2), (24, 256, 128, 7)]
TOKENS = [1, 2, 8, 9, 16, 17, 40, 65]


@pytest.mark.parametrize("E,H,F,top_k", SHAPES)
@pytest.mark.parametrize("K,Kd", [(1, 1), (2, 2), (3, 3), (4, 4), (2, 3), (4, 1)])
@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_layer(ex, E, H, F, top_k, K, Kd, tr, dt):
    g = gen(E + K)
    m = Experts(g, E, H, F, K, Kd, tr)
    for T in TOKENS:
        x, router = acts(g, T, H, dt), a_router(g, E, H, DT[dt])
        y = m.run(ex, x, top_k, router=router)
        assert y.shape == (T, H) and y.dtype is DT[dt]
        within(y, expected(m, x, *picks(x, router, top_k), dt))


@pytest.mark.parametrize("T", [3, 100, 256])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_many_experts_and_picks(ex, T, dt):
    """More experts than the picks keep in registers, more tiles than a block's table."""
    g = gen(T)
    m = Experts(g, 200, 128, 128, 2, 2, False)
    x, router = acts(g, T, 128, dt), a_router(g, 200, 128, torch.float32)
    top_k = 16 if T == 256 else 32
    within(m.run(ex, x, top_k, router=router), expected(m, x, *picks(x, router, top_k), dt))
    within(m.run(ex, x, 3, router=router, normalize=False), expected(m, x, *picks(x, router, 3, False), dt))


def test_a_thousand_experts(ex):
    g = gen(12)
    m = Experts(g, 1024, 128, 128, 1, 1, False)
    for T, top_k in ((2, 3), (40, 1)):
        x, router = acts(g, T, 128, "bf16"), a_router(g, 1024, 128, torch.bfloat16)
        within(m.run(ex, x, top_k, router=router), expected(m, x, *picks(x, router, top_k), "bf16"))
    ids = torch.randint(0, 1024, (256, 16), generator=g, device=DEV, dtype=torch.int32)
    w = torch.rand(256, 16, generator=g, device=DEV)
    x = acts(g, 256, 128, "bf16")
    y = m.run(ex, x, 16, ids=ids, weights=w)
    part = m.run(ex, x[100:103], 16, ids=ids[100:103].contiguous(), weights=w[100:103].contiguous())
    within(part, expected(m, x[100:103], ids[100:103], w[100:103], "bf16"))
    assert float((y[100:103].float() - part.float()).norm()) <= 2.0 ** -7 * float(part.float().norm())


@pytest.mark.parametrize("H,F,tr", [(17408, 128, False), (128, 16512, True), (4096, 1152, True)])
def test_long_sides(ex, H, F, tr):
    g = gen(H)
    m = Experts(g, 2, H, F, 3, 2, tr)
    for T in (1, 20):
        x, router = acts(g, T, H, "bf16"), a_router(g, 2, H, torch.bfloat16)
        within(m.run(ex, x, 1, router=router), expected(m, x, *picks(x, router, 1), "bf16"))


def test_equal_logits_pick_the_first(ex):
    """Experts with the same router row stand in their order."""
    for E, top_k in ((40, 5), (70, 9)):
        g = gen(E)
        m = Experts(g, E, 128, 128, 2, 2, False)
        x, router = acts(g, 6, 128, "bf16"), torch.zeros(E, 128, device=DEV)
        within(m.run(ex, x, top_k, router=router), expected(m, x, *picks(x, router, top_k), "bf16"))
        router = a_router(g, E, 128, torch.float32)
        router[E // 2:] = router[:E - E // 2].clone()
        within(m.run(ex, x, top_k, router=router), expected(m, x, *picks(x, router, top_k), "bf16"))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 5, 30, 256])
def test_given_picks(ex, T, dt):
    """Ids that are none, the same expert twice, tokens without any, all tokens at one expert."""
    g = gen(T)
    E, H, F, k = 12, 256, 384, 4
    m = Experts(g, E, H, F, 2, 4, True)
    x = acts(g, T, H, dt)
    w = torch.randn(T, k, generator=g, device=DEV)
    some = torch.randint(-3, E + 3, (T, k), generator=g, device=DEV, dtype=torch.int32)
    some[T // 2] = -1
    some[0, :2] = 7
    for ids in (some, torch.full_like(some, 5), torch.full_like(some, E), torch.full_like(some, 2 ** 31 - 1)):
        valid = torch.where((ids >= 0) & (ids < E), ids, -1)
        y = m.run(ex, x, k, ids=ids, weights=w)
        within(y, expected(m, x, valid, w, dt))
        assert bool((y[(valid < 0).all(1)] == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_strided_rows_and_results_into_columns(ex, dt):
    g = gen(4)
    E, H, F, T, k = 6, 384, 256, 21, 3
    m = Experts(g, E, H, F, 3, 2, False)
    x, router = acts(g, T, H, dt), a_router(g, E, H, DT[dt])
    want = expected(m, x, *picks(x, router, k), dt)
    for at in (0, 5, 8):
        buf = torch.full((T, H + 40), 7.0, dtype=DT[dt], device=DEV)
        buf[:, at:at + H] = x
        out = torch.full((T, H + 40), 3.0, dtype=DT[dt], device=DEV)
        y = m.run(ex, buf[:, at:at + H], k, router=router, out=out[:, at:at + H])
        assert y.data_ptr() == out[:, at:].data_ptr()
        within(out[:, at:at + H], want)
        assert bool((out[:, :at] == 3).all()) and bool((out[:, at + H:] == 3).all())


@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_tokens_stay_apart(ex, value):
    g = gen(6)
    E, H, F, T, k = 9, 256, 256, 19, 3
    m = Experts(g, E, H, F, 2, 2, False)
    x, router = acts(g, T, H, "bf16"), a_router(g, E, H, torch.bfloat16)
    ids, w = picks(x, router, k)
    ids, w = ids.int(), w.float().contiguous()
    bad = x.clone()
    bad[4, 100] = value
    y0, y1 = m.run(ex, x, k, ids=ids, weights=w), m.run(ex, bad, k, ids=ids, weights=w)
    keep = torch.arange(T, device=DEV) != 4
    assert torch.equal(y0[keep], y1[keep]) and not bool(y1[4].float().isfinite().any())
    # its logits are no numbers either: some experts, and the other tokens' results within tolerance
    y2 = m.run(ex, bad, k, router=router)
    y, tol = expected(m, x, *picks(x, router, k), "bf16")
    within(y2[keep], (y[keep], tol[keep]))


def test_large_and_small_activations(ex):
    """x's range is taken out before anything is rounded to binary16 (a token of zeros among them)."""
    g = gen(7)
    m = Experts(g, 4, 256, 128, 2, 2, False)
    x = acts(g, 6, 256, "bf16")
    x *= torch.tensor([1.0, 1e3, 1e-3, 0.0, 1e-6, 30.0], device=DEV).bfloat16()[:, None]
    ids = torch.arange(6, device=DEV, dtype=torch.int32)[:, None] % 4
    w = torch.ones(6, 1, device=DEV)
    y = m.run(ex, x, 1, ids=ids, weights=w)
    within(y, expected(m, x, ids, w, "bf16"))
    assert bool((y[3] == 0).all())


def test_same_results_with_any_workspace_graph_and_stream(ex):
    g = gen(8)
    E, H, F, T, k = 16, 256, 384, 24, 4
    m = Experts(g, E, H, F, 2, 2, False)
    x, router = acts(g, T, H, "bf16"), a_router(g, E, H, torch.bfloat16)
    ws = torch.full((ex.expert_layer_workspace_bytes(T, H, F, E, k),), 255, dtype=torch.uint8, device=DEV)
    want = m.run(ex, x, k, router=router)
    for _ in range(20):
        assert torch.equal(m.run(ex, x, k, router=router, ws=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = m.run(ex, x, k, router=router)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    # two graphs with one workspace, replayed one after the other with other tokens
    x2 = acts(g, T, H, "bf16")
    graphs = []
    for v in (x, x2):
        q = torch.cuda.CUDAGraph()
        with torch.cuda.graph(q):
            y = m.run(ex, v, k, router=router, ws=ws)
        graphs.append((q, v, y))
    for i in range(4):
        for q, v, y in graphs:
            v.copy_(acts(g, T, H, "bf16"))
            q.replay()
        for q, v, y in graphs[1:]:
            assert torch.equal(y, m.run(ex, v, k, router=router))
    # calls on two streams at once, each with its own workspace
    ys = [m.run(ex, v, k, router=router) for v in (x, x2)]
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            a = m.run(ex, x, k, router=router)
        b = m.run(ex, x2, k, router=router)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, ys[0]) and torch.equal(b, ys[1])


def test_without_tokens(ex):
    g = gen(9)
    m = Experts(g, 3, 128, 128, 2, 2, False)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    assert m.run(ex, x, 2, router=a_router(g, 3, 128, torch.bfloat16)).shape == (0, 128)


def test_refusals(ex):
    g = gen(10)
    m = Experts(g, 3, 128, 256, 2, 2, False)
    x, router = acts(g, 4, 128, "bf16"), a_router(g, 3, 128, torch.bfloat16)
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.ones(4, 2, device=DEV)
    for kw in (dict(), dict(router=router, ids=ids, weights=w), dict(ids=ids), dict(ids=ids.long(), weights=w),
               dict(router=router.half()), dict(router=router[:2]), dict(router=router[:, ::2]), dict(router=router.cpu()),
               dict(router=router, out=torch.empty(3, 128, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ValueError):
            m.run(ex, x, 2, **kw)
    with pytest.raises(ValueError, match="no gradient"):
        m.run(ex, x.clone().requires_grad_(), 2, router=router)
    with torch.no_grad():
        m.run(ex, x.clone().requires_grad_(), 2, router=router)
    with pytest.raises(ex.Exl3Error, match="picks"):
        m.run(ex, x, 4, router=router)
    with pytest.raises(ex.Exl3Error, match="tokens"):
        m.run(ex, acts(g, 257, 128, "bf16"), 2, router=router)
    with pytest.raises(ValueError, match="go together"):
        ex.expert_layer(x, m.gate, m.up, m.gate, 2, 2, router=router)
    with pytest.raises(ex.Exl3Error, match="overlaps"):
        m.run(ex, x, 2, router=router, out=x)


def test_a_layer_of_them_together(ex):
    """Residual, norm, experts and an 8-bit projection as a decoding step uses them, in a graph:
    the same as its parts, and as the products grouped by expert up to their roundings."""
    g = gen(11)
    E, H, F, T, k = 8, 512, 256, 6, 2
    m = Experts(g, E, H, F, 2, 2, False)
    x, r, router = acts(g, T, H, "bf16"), acts(g, T, H, "bf16"), a_router(g, E, H, torch.bfloat16)
    w1, w2 = torch.rand(H, generator=g, device=DEV) + 0.5, torch.rand(H, generator=g, device=DEV) + 0.5
    w8, s8 = ex.quantize8(torch.randn(H, 768, generator=g, device=DEV), block_rows=128)

    def step():
        a = ex.rms_norm(x, w1, residual=r)
        y = m.run(ex, a["y"], k, router=router)
        b = ex.rms_norm(y, w2, residual=a["h"], want_y=False, want_y8=True)
        return a["y"], y, b["h"], ex.linear8(b["y8"], w8, s8, b["scale"])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(acts(g, T, H, "bf16"))
    graph.replay()
    assert all(torch.equal(p, q) for p, q in zip(got, step()))
    a, y, h, z = got
    ids, w = picks(a, router, k)
    within(y, expected(m, a, ids, w, "bf16"))
    # the same picks through expert_linear, whose results are rounded to bfloat16 between the products
    order = torch.argsort(ids.flatten(), stable=True)
    off = torch.cat([torch.zeros(1, device=DEV), torch.bincount(ids.flatten(), minlength=E).cumsum(0)]).int()
    rows = a[order // k]
    p, q = (ex.expert_linear(rows, off, *t[:3], 2, t[3]) for t in (m.gate, m.up))
    parts = ex.expert_linear((torch.nn.functional.silu(p.float()) * q.float()).bfloat16(), off, *m.down[:3], 2, m.down[3])
    other = torch.zeros(T, H, device=DEV).index_add_(0, order // k, parts.float() * w.flatten()[order].float()[:, None])
    assert float((other - y.float()).norm()) <= 4 * 2.0 ** -8 * float(y.float().norm())
    W = w8.double() * s8.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    v = h.double() / torch.sqrt(h.double().pow(2).mean(1, keepdim=True) + 1e-6) * w2.double()
    # e4m3 rounds by 2^-4 at most, 2^-4 / sqrt(3) in the root mean square, of each input on its own
    tol = 6 * 2.0 ** -4 / math.sqrt(3) * (v.pow(2) @ W.pow(2)).sqrt() + 2.0 ** -8 * (v @ W).abs()
    assert bool(((z.double() - v @ W).abs() <= tol).all())
