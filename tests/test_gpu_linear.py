"""Products with trellis-coded matrices on the GPU, against the definition in
64 bits.

Tolerances.  The rotated activations are rounded to binary16 (relative error of
each at most 2^-11, independent), everything after that is binary32 up to the
one rounding of the result (2^-8 for bfloat16, 2^-11 for float16, of each value
itself).  The rotations keep norms, so before the channel factor `right` the
first error has a standard deviation below 2^-11 / sqrt(3) of the row's root
mean square in every channel: six of those are far outside of what chance gives.
Adapter terms are products of values rounded at most once to the inputs' type on
the way (u = 2^-8 or 2^-11), and their errors are held to six times u / sqrt(3)
of the row's adapter term plus the same of a token's adapter sums.  Gradients of
A and B are sums over tokens of such terms.  A float16 result below the smallest
normal number, 2^-14, may be off by half a subnormal step, 2^-25.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import oracle  # noqa: E402

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


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


def coded(g, rows, cols, K, lead=()):
    codes = torch.randint(-32768, 32768, (*lead, rows // 16, cols // 16, 16 * K), generator=g, device=DEV,
                          dtype=torch.int32).to(torch.int16)
    su = (torch.randint(0, 2, (*lead, rows), generator=g, device=DEV) * 2 - 1).float()
    sv = (torch.randint(0, 2, (*lead, cols), generator=g, device=DEV) * 2 - 1).float()
    sv *= 0.05 * torch.exp(0.5 * torch.randn(*lead, cols, generator=g, device=DEV))
    sv[..., 5] = 0.0
    scale = (0.5 + torch.rand(lead, generator=g, device=DEV)) if lead else torch.tensor(0.75, device=DEV)
    return codes, su, sv, scale


def weight64(codes, su, sv, K, scale):
    """The decoded matrix from the oracle's codebook and packing, rotated back densely in 64 bits."""
    R, C, n = codes.shape
    words = codes.cpu().numpy().view(np.uint16).reshape(-1, n)
    stream = words.reshape(-1, 8 * K, 2)[:, :, ::-1].reshape(-1, 16 * K)
    bits = np.unpackbits(stream.astype(">u2").view(np.uint8).reshape(len(words), -1), axis=1)
    ext = np.concatenate([bits[:, -16:], bits], axis=1).astype(np.int64)
    state = np.zeros((len(words), 256), dtype=np.int64)
    for b in range(16):
        at = 16 + (np.arange(256) + 1) * K - 16 + b
        state |= ext[:, at] << (15 - b)
    table = oracle.mul1_table().astype(np.float64)
    V = table[state].reshape(R, C, 16, 16).transpose(0, 2, 1, 3).reshape(R * 16, C * 16)
    V = torch.from_numpy(V).to(DEV)
    H = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    for _ in range(7):
        H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)], 0)
    V = (H @ V.view(R // 8, 128, C * 16)).view(R * 16, C * 16)
    V = (V.view(R * 16, C // 8, 128) @ H).reshape(R * 16, C * 16)
    return V * su.double()[:, None] * sv.double()[None, :] * float(scale) / 128.0


def close(y, ref, right, dt, base=None, extra=None):
    """|y - ref| within the rounding of y, the rounding of the rotated activations
    (of the rows of `base`, the part of ref that comes from the coded matrix) and
    `extra` (of the adapters)."""
    y, base = y.double(), ref if base is None else base
    live = right != 0
    rms = torch.zeros(y.shape[0], 1, dtype=torch.float64, device=y.device)
    if live.any():
        rms = (base[:, live] / right[live]).pow(2).mean(1, keepdim=True).sqrt()
    tol = U[dt] * ref.abs() + 2.0 ** -25 + 6 * 2.0 ** -11 / math.sqrt(3) * rms * right.abs()
    if extra is not None:
        tol = tol + extra
    bad = ~((y - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((y - ref).abs() / tol).max()))


def acts(g, T, n, dt, scale=1.0):
    x = torch.randn(T, n, generator=g, device=DEV) * scale
    x[:, 3] *= 15.0
    return x.to(DT[dt])


def adapters(g, n, r, n_in, n_out, dt):
    A = (torch.randn(n, r, n_in, generator=g, device=DEV) / math.sqrt(n_in)).to(DT[dt])
    B = (torch.randn(n, r, n_out, generator=g, device=DEV) * 0.5).to(DT[dt])
    gain = 0.25 + torch.rand(n, generator=g, device=DEV)
    ranks = torch.randint(0, r + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    return A, B, gain, ranks


def adapter64(x, A, B, gain, slots, ranks):
    """(term [T, outputs], its error scale [T, 1] per unit roundoff)."""
    y = torch.zeros(x.shape[0], B.shape[2], dtype=torch.float64, device=x.device)
    e = torch.zeros_like(y)
    for i in range(A.shape[0]):
        t = torch.nonzero(slots == i).flatten()
        r = A.shape[1] if ranks is None else int(ranks[i].clamp(0, A.shape[1]))
        h = float(gain[i]) * (x[t].double() @ A[i, :r].double().t())
        y[t] = h @ B[i, :r].double()
        e[t] = (h.pow(2) @ B[i, :r].double().pow(2)).sqrt()      # root sum of the terms' squares
    return y, e


TOKENS = [1, 2, 7, 8, 9, 16, 17, 33, 64, 100, 255, 256, 257, 300, 513, 777]
SIZES = [(128, 128), (256, 128), (128, 384), (640, 256), (1152, 1280)]


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_linear_every_size(ex, K, tr, dt):
    for s, (rows, cols) in enumerate(SIZES):
        g = gen(100 * K + 10 * s + tr)
        codes, su, sv, scale = coded(g, rows, cols, K)
        W = weight64(codes, su, sv, K, scale)
        W = W.t() if tr else W
        right = (su if tr else sv).double()
        for T in TOKENS if s in (0, 4) else TOKENS[s::4]:
            x = acts(g, T, W.shape[0], dt)
            y = ex.linear(x, codes, su, sv, K, scale, transposed=tr)
            assert y.shape == (T, W.shape[1]) and y.dtype == x.dtype
            close(y, x.double() @ W, right, dt)


def test_linear_matches_the_library_decode(ex):
    """The same matrix as exl3_decode_tiles and the inverse rotation give."""
    g = gen(5)
    codes, su, sv, scale = coded(g, 256, 384, 3)
    W = ex.rotate(ex.decode_tiles(codes, 256, 384, 3, float(scale)), su, sv, inverse=True)
    x = acts(g, 40, 256, "bf16")
    close(ex.linear(x, codes, su, sv, 3, scale), x.double() @ W.double(), sv.double(), "bf16")
    # a number for the scale is the same call
    assert torch.equal(ex.linear(x, codes, su, sv, 3, scale), ex.linear(x, codes, su, sv, 3, float(scale)))


@pytest.mark.parametrize("rows,cols,T", [(4096, 1024, 3), (1024, 8192, 130), (2048, 2048, 1100)])
def test_linear_long_sums(ex, rows, cols, T):
    g = gen(rows + T)
    codes, su, sv, scale = coded(g, rows, cols, 2)
    W = weight64(codes, su, sv, 2, scale)
    for tr in (False, True):
        M = W.t() if tr else W
        x = acts(g, T, M.shape[0], "fp16")
        close(ex.linear(x, codes, su, sv, 2, scale, transposed=tr), x.double() @ M, (su if tr else sv).double(), "fp16")


def test_linear_strided_and_unaligned_rows(ex):
    g = gen(9)
    codes, su, sv, scale = coded(g, 256, 384, 2)
    W = weight64(codes, su, sv, 2, scale)
    for T in (1, 5, 70, 300):
        for off, pad in ((64, 192), (1, 3), (8, 8), (4, 12)):
            buf = torch.full((T, 256 + off + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
            x = buf[:, off:off + 256]
            x.copy_(acts(g, T, 256, "bf16"))
            whole = torch.full((T, 384 + off + pad), 7.0, dtype=torch.bfloat16, device=DEV)
            out = whole[:, off:off + 384]
            y = ex.linear(x, codes, su, sv, 2, scale, out=out)
            assert y is out
            close(out, x.double() @ W, sv.double(), "bf16")
            assert (whole[:, :off] == 7.0).all() and (whole[:, off + 384:] == 7.0).all()


def test_python_refusals(ex):
    g = gen(8)
    codes, su, sv, scale = coded(g, 256, 128, 2)
    x = acts(g, 3, 256, "bf16")
    A, B, gain, ranks = adapters(g, 2, 4, 256, 128, "bf16")
    slots = torch.zeros(3, dtype=torch.int32, device=DEV)
    ok = dict(A=A, B=B, gain=gain, slots=slots, ranks=ranks)
    ex.linear(x, codes, su, sv, 2, scale, **ok)
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(x=x.t().contiguous().t()), dict(x=x[:1].t().repeat(1, 2)[:, :1].t()),
                dict(x=x.cpu()), dict(su=su.cpu()), dict(sv=sv.double()), dict(scale=scale.double()),
                dict(A=A.half()), dict(A=A[0]), dict(B=B[:, :2]), dict(B=None), dict(gain=gain[:1]), dict(slots=slots.long()),
                dict(slots=slots[:2]), dict(ranks=ranks.float()), dict(A=None), dict(out=torch.empty(3, 128, device=DEV)),
                dict(out=torch.empty(2, 128, dtype=torch.bfloat16, device=DEV))):
        kw = dict(x=x, codes=codes, su=su, sv=sv, K=2, scale=scale, **ok)
        kw.update(bad)
        with pytest.raises(ValueError):
            ex.linear(**kw)
    with pytest.raises(ex.Exl3Error) as e:
        ex.linear(x, codes, su, sv, 2, scale, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == 3
    with pytest.raises(ex.Exl3Error) as e:
        buf = torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV)
        ex.linear(buf, codes, su, sv, 2, scale, out=buf[:, :128])
    assert e.value.status == 1
    with pytest.raises(ValueError):
        ex.linear_backward(acts(g, 3, 128, "bf16"), None, codes, su, sv, 2, scale, **ok)
    with pytest.raises(ValueError):
        ex.expert_linear(x, torch.zeros(3, dtype=torch.int32, device=DEV), codes[None], su[None], sv[None], 2, scale[None])


def test_linear_row_ranges_and_special_values(ex):
    """Rows of zeros, of very large and very small values; rows that are not numbers stay alone."""
    g = gen(10)
    codes, su, sv, scale = coded(g, 256, 256, 4)
    W = weight64(codes, su, sv, 4, scale)
    for T in (6, 40):
        x = acts(g, T, 256, "bf16")
        x[0] = 0
        x[1] *= 1e30
        x[2] *= 1e-30
        x[3, 17] = float("inf")
        x[4, 200] = float("nan")
        y = ex.linear(x, codes, su, sv, 4, scale)
        ok = torch.ones(T, dtype=torch.bool, device=DEV)
        ok[3:5] = False
        assert (y[0] == 0).all()
        assert torch.isfinite(y[ok]).all()
        live = sv != 0
        assert not torch.isfinite(y[3:5][:, live]).any()
        close(y[ok], x[ok].double() @ W, sv.double(), "bf16")


def test_linear_without_tokens(ex):
    g = gen(11)
    codes, su, sv, scale = coded(g, 128, 256, 2)
    x = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    assert ex.linear(x, codes, su, sv, 2, scale).shape == (0, 256)
    A, B, gain, _ = adapters(g, 2, 4, 128, 256, "bf16")
    slots = torch.empty(0, dtype=torch.int32, device=DEV)
    dy = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    gr = ex.linear_backward(dy, x, codes, su, sv, 2, scale, A=A, B=B, gain=gain, slots=slots)
    assert gr["dx"].shape == (0, 128) and (gr["dA"] == 0).all() and (gr["dB"] == 0).all()


def _slots(g, how, T, n):
    if how == "mixed":            # out of range on both sides, one adapter unused
        return torch.randint(-2, n + 1, (T,), generator=g, device=DEV, dtype=torch.int32).where(
            torch.rand(T, generator=g, device=DEV) < 0.9, torch.tensor(-7, dtype=torch.int32, device=DEV))
    if how == "one":
        return torch.full((T,), n - 1, dtype=torch.int32, device=DEV)
    if how == "none":
        return torch.full((T,), -1, dtype=torch.int32, device=DEV)
    return (torch.arange(T, device=DEV) * n // max(T, 1)).int()      # runs


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("how", ["mixed", "one", "none", "runs"])
def test_adapters_forward(ex, dt, how):
    for s, (T, n, r, tr) in enumerate([(1, 1, 1, False), (5, 3, 16, True), (33, 40, 7, False), (64, 4, 64, True),
                                       (200, 9, 128, False), (600, 5, 20, True), (1500, 300, 12, False)]):
        g = gen(1000 + s)
        codes, su, sv, scale = coded(g, 384, 640, 2)
        W = weight64(codes, su, sv, 2, scale)
        W = W.t() if tr else W
        A, B, gain, ranks = adapters(g, n, r, W.shape[0], W.shape[1], dt)
        slots = _slots(g, how, T, n)
        x = acts(g, T, W.shape[0], dt)
        for rk in (ranks, None):
            y = ex.linear(x, codes, su, sv, 2, scale, transposed=tr, A=A, B=B, gain=gain, slots=slots, ranks=rk)
            term, err = adapter64(x, A, B, gain, slots, rk)
            base = x.double() @ W
            close(y, base + term, (su if tr else sv).double(), dt, base, 6 * U[dt] / math.sqrt(3) * err)


def test_adapter_rows_behind_the_rank_are_not_read(ex):
    g = gen(12)
    codes, su, sv, scale = coded(g, 256, 256, 2)
    for T in (4, 90, 700):
        A, B, gain, _ = adapters(g, 3, 24, 256, 256, "bf16")
        ranks = torch.tensor([24, 5, 0], dtype=torch.int32, device=DEV)
        slots = (torch.arange(T, device=DEV) % 3).int()
        x, dy = acts(g, T, 256, "bf16"), acts(g, T, 256, "bf16")
        Z, Y = A.clone(), B.clone()
        for i in range(3):
            Z[i, ranks[i]:], Y[i, ranks[i]:] = float("nan"), float("inf")
        kw = dict(gain=gain, slots=slots, ranks=ranks)
        assert torch.equal(ex.linear(x, codes, su, sv, 2, scale, A=A, B=B, **kw),
                           ex.linear(x, codes, su, sv, 2, scale, A=Z, B=Y, **kw))
        p = ex.linear_backward(dy, x, codes, su, sv, 2, scale, A=A, B=B, **kw)
        q = ex.linear_backward(dy, x, codes, su, sv, 2, scale, A=Z, B=Y, **kw)
        for k in p:
            assert torch.equal(p[k], q[k])
        for i in range(3):
            assert (p["dA"][i, ranks[i]:] == 0).all() and (p["dB"][i, ranks[i]:] == 0).all()


def _grad_close(got, ref, err, dt):
    tol = U[dt] * ref.abs() + 2.0 ** -25 + 6 * U[dt] / math.sqrt(3) * err
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - ref).abs() / tol).max()))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("how", ["mixed", "one", "runs"])
def test_backward_against_the_formulas(ex, dt, how):
    for s, (T, n, r, tr) in enumerate([(1, 2, 3, False), (17, 5, 16, True), (96, 3, 8, True), (130, 2, 100, False),
                                       (1001, 5, 12, False), (2100, 70, 64, True)]):
        g = gen(2000 + s)
        codes, su, sv, scale = coded(g, 384, 640, 3)
        W = weight64(codes, su, sv, 3, scale)
        W = W.t() if tr else W
        A, B, gain, ranks = adapters(g, n, r, W.shape[0], W.shape[1], dt)
        slots = _slots(g, how, T, n)
        x, dy = acts(g, T, W.shape[0], dt), acts(g, T, W.shape[1], dt, 0.1)
        got = ex.linear_backward(dy, x, codes, su, sv, 3, scale, transposed=tr, A=A, B=B, gain=gain, slots=slots,
                                 ranks=ranks)
        term, err = adapter64(dy, B, A, gain, slots, ranks)
        base = dy.double() @ W.t()
        close(got["dx"], base + term, (sv if tr else su).double(), dt, base, 6 * U[dt] / math.sqrt(3) * err)
        for i in range(n):
            t, k = torch.nonzero(slots == i).flatten(), int(ranks[i])
            a, X, D = float(gain[i]), x[t].double(), dy[t].double()
            gg, h = a * (D @ B[i, :k].double().t()), a * (X @ A[i, :k].double().t())
            for name, p, q in (("dA", gg, X), ("dB", h, D)):
                _grad_close(got[name][i, :k], p.t() @ q, (p.pow(2).t() @ q.pow(2)).sqrt(), dt)
                assert (got[name][i, k:] == 0).all()


def test_backward_against_differences(ex):
    """The loss sum(y . c) is linear in x, in A and in B: differences of the forward's
    results in 64 bits of its inputs' roundings are exact up to the results' rounding."""
    g = gen(31)
    T, n, r = 20, 2, 4
    codes, su, sv, scale = coded(g, 256, 128, 2)
    A, B, gain, _ = adapters(g, n, r, 256, 128, "fp16")
    slots = torch.randint(-1, n, (T,), generator=g, device=DEV, dtype=torch.int32)
    x, c = acts(g, T, 256, "fp16"), acts(g, T, 128, "fp16", 0.25)
    kw = dict(gain=gain, slots=slots)

    def loss(x, A, B):
        return (ex.linear(x, codes, su, sv, 2, scale, A=A, B=B, **kw).double() * c.double()).sum()

    gr = ex.linear_backward(c, x, codes, su, sv, 2, scale, A=A, B=B, **kw)
    y = ex.linear(x, codes, su, sv, 2, scale, A=A, B=B, **kw).double()
    for name, at in (("x", 0), ("A", 1), ("B", 2)):
        args = [x, A, B]
        d = torch.randn(args[at].shape, generator=g, device=DEV).to(torch.float16)
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + d, args[at] - d
        step = (up[at].double() - dn[at].double())
        grad = gr["d" + name].double()
        want = (loss(*up) - loss(*dn))
        got = (grad * step).sum()
        # independent roundings of y+ and y- (with the activations') and of the gradient, six deviations
        big = max(y.abs().max(), ex.linear(*[up[0]], codes, su, sv, 2, scale, A=up[1], B=up[2], **kw).double().abs().max())
        tol = 6 * 2 * 2.0 ** -11 * (float(big) * float(c.double().norm()) * 2 + float((grad * step).norm()))
        assert abs(float(want - got)) <= tol, (name, float(want), float(got), tol)


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("tr", [False, True])
def test_experts_ragged(ex, K, tr):
    rows, cols = 384, 256
    for s, counts in enumerate([[3], [0, 0, 5, 0], [1, 0, 7, 8, 9, 0, 64, 31], [300, 0, 17, 600], [1] * 33,
                                [0] * 100 + [2, 0, 1], [256, 255, 257]]):
        g = gen(3000 + 10 * s + K)
        E = len(counts)
        dt = "bf16" if s % 2 else "fp16"
        codes, su, sv, scale = coded(g, rows, cols, K, (E,))
        off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
        T = int(off[-1])
        x = acts(g, T, cols if tr else rows, dt)
        y = ex.expert_linear(x, off, codes, su, sv, K, scale, transposed=tr)
        for e, m in enumerate(counts):
            if m:
                a = int(off[e])
                W = weight64(codes[e], su[e], sv[e], K, scale[e])
                close(y[a:a + m], x[a:a + m].double() @ (W.t() if tr else W), (su if tr else sv)[e].double(), dt)


def test_experts_rows_of_no_expert_are_zero(ex):
    g = gen(40)
    codes, su, sv, scale = coded(g, 128, 256, 2, (3,))
    off = torch.tensor([5, 9, 9, 30], dtype=torch.int32, device=DEV)
    for T in (33, 30):
        x = acts(g, T, 128, "bf16")
        out = torch.full((T, 256 + 8), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :256]
        y = ex.expert_linear(x, off, codes, su, sv, 2, scale, out=out)
        assert (y[:5] == 0).all() and (y[30:] == 0).all()
        for e, (a, b) in enumerate([(5, 9), (9, 9), (9, 30)]):
            if b > a:
                close(y[a:b], x[a:b].double() @ weight64(codes[e], su[e], sv[e], 2, scale[e]), sv[e].double(), "bf16")
    none = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert (ex.expert_linear(x, none, codes, su, sv, 2, scale) == 0).all()


def test_one_expert_is_linear(ex):
    g = gen(41)
    codes, su, sv, scale = coded(g, 256, 256, 3, (1,))
    x = acts(g, 300, 256, "fp16")
    off = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    assert torch.equal(ex.expert_linear(x, off, codes, su, sv, 3, scale),
                       ex.linear(x, codes[0], su[0], sv[0], 3, scale[0]))


def test_same_results_on_another_stream_and_again(ex):
    g = gen(42)
    codes, su, sv, scale = coded(g, 1024, 512, 2)
    A, B, gain, ranks = adapters(g, 6, 16, 1024, 512, "bf16")
    for T in (3, 70, 900):
        x, dy = acts(g, T, 1024, "bf16"), acts(g, T, 512, "bf16")
        slots = torch.randint(-1, 6, (T,), generator=g, device=DEV, dtype=torch.int32)
        kw = dict(A=A, B=B, gain=gain, slots=slots, ranks=ranks)
        first = [ex.linear(x, codes, su, sv, 2, scale, **kw), *ex.linear_backward(dy, x, codes, su, sv, 2, scale, **kw).values()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = [ex.linear(x, codes, su, sv, 2, scale, **kw),
                     *ex.linear_backward(dy, x, codes, su, sv, 2, scale, **kw).values()]
        side.synchronize()
        for p, q in zip(first, again):
            assert torch.equal(p, q)


def test_workspace_contents_do_not_matter(ex):
    """Rows of padding inside the workspace may hold anything."""
    g = gen(43)
    codes, su, sv, scale = coded(g, 256, 256, 2)
    for T in (1, 13, 290):
        x = acts(g, T, 256, "bf16")
        need = ex.linear_workspace_bytes(T, 256, 256)
        outs = []
        for fill in (0, 255):
            ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
            outs.append(ex.linear(x, codes, su, sv, 2, scale, ws=ws))
        assert torch.equal(*outs)


def test_capture_in_a_graph(ex):
    g = gen(44)
    codes, su, sv, scale = coded(g, 512, 256, 2)
    A, B, gain, ranks = adapters(g, 4, 8, 512, 256, "bf16")
    slots = torch.tensor([0, 3, -1, 2], dtype=torch.int32, device=DEV)
    x = acts(g, 4, 512, "bf16")
    kw = dict(A=A, B=B, gain=gain, slots=slots, ranks=ranks, out=torch.empty(4, 256, dtype=torch.bfloat16, device=DEV),
              ws=torch.empty(ex.linear_workspace_bytes(4, 512, 256, False, 4, 8), dtype=torch.uint8, device=DEV))
    want = ex.linear(x, codes, su, sv, 2, scale, **kw).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex.linear(x, codes, su, sv, 2, scale, **kw)
    kw["out"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kw["out"], want)


def test_calls_back_to_back_in_one_workspace(ex):
    """A call's kernels overlap one another, not those of the calls around it."""
    g = gen(45)
    codes, su, sv, scale = coded(g, 512, 1024, 3)
    A, B, gain, ranks = adapters(g, 5, 48, 512, 1024, "bf16")
    T = 700
    sets = []
    for _ in range(3):
        x, dy = acts(g, T, 512, "bf16"), acts(g, T, 1024, "bf16")
        slots = torch.randint(-1, 5, (T,), generator=g, device=DEV, dtype=torch.int32)
        sets.append((x, dy, dict(A=A, B=B, gain=gain, slots=slots, ranks=ranks)))
    ws = torch.empty(ex.linear_backward_workspace_bytes(T, 512, 1024, False, 5, 48), dtype=torch.uint8, device=DEV)

    def call(x, dy, kw):
        return [ex.linear(x, codes, su, sv, 3, scale, ws=ws, **kw),
                *ex.linear_backward(dy, x, codes, su, sv, 3, scale, ws=ws, **kw).values()]

    want = []
    for s in sets:
        want.append(call(*s))
        torch.cuda.synchronize()
    got = [call(*sets[i % 3]) for i in range(30)]
    for i, outs in enumerate(got):
        for p, q in zip(outs, want[i % 3]):
            assert torch.equal(p, q)


def test_backward_capture_in_a_graph(ex):
    g = gen(46)
    codes, su, sv, scale = coded(g, 256, 384, 2)
    A, B, gain, ranks = adapters(g, 4, 16, 256, 384, "fp16")
    for T in (20, 200):
        x, dy = acts(g, T, 256, "fp16"), acts(g, T, 384, "fp16")
        slots = torch.randint(-1, 4, (T,), generator=g, device=DEV, dtype=torch.int32)
        kw = dict(A=A, B=B, gain=gain, slots=slots, ranks=ranks)
        want = ex.linear_backward(dy, x, codes, su, sv, 2, scale, **kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = ex.linear_backward(dy, x, codes, su, sv, 2, scale, **kw)
        for _ in range(3):
            for t in got.values():
                t.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            for k in want:
                assert torch.equal(got[k], want[k])


def test_the_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "coded_layer.py")
    spec = importlib.util.spec_from_file_location("coded_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.main()
