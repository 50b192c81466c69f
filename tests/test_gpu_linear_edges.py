"""Products with trellis-coded matrices on the GPU where they can go wrong: values far
apart, rows that are not numbers, the forms that only large sizes reach.

References, inputs and `close` are those of test_gpu_linear.py (64 bits; six standard
deviations of the rounding of the rotated activations, one rounding of the result)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_linear import (DEV, U, _no_expired_waits, acts, adapter64, adapters, close, coded, ex,  # noqa: E402,F401
                             gen, weight64)


def test_adapters_of_a_token_do_not_depend_on_its_neighbours(ex):
    """float16, tokens sorted into tiles by adapter: an infinite row, sums beyond binary16's
    range and sums a hundred million times smaller side by side.  The coded part is small, so
    that what is left of an adapter's term shows."""
    g = gen(51)
    codes, su, sv, scale = coded(g, 256, 384, 2)
    scale = scale * 1e-6
    W = weight64(codes, su, sv, 2, scale)
    for T in (65, 200):
        x = torch.randn(T, 256, generator=g, device=DEV)
        size = torch.tensor([1e4, 1.0, 1e-4, 30.0], device=DEV)[torch.arange(T, device=DEV) % 4]
        x = (x * size[:, None]).half()
        A = (100 * torch.randn(1, 4, 256, generator=g, device=DEV)).half()
        B = (2e-4 * torch.randn(1, 4, 384, generator=g, device=DEV)).half()
        gain, slots = torch.ones(1, device=DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
        kw = dict(A=A, B=B, gain=gain, slots=slots)
        y = ex.linear(x, codes, su, sv, 2, scale, **kw)
        term, err = adapter64(x, A, B, gain, slots, None)
        assert (torch.mm(x.float(), A[0].float().t()).abs() > 65504).any()
        base = x.double() @ W
        close(y, base + term, sv.double(), "fp16", base, 6 * U["fp16"] / math.sqrt(3) * err)
        bad = x.clone()
        bad[5, 17] = float("inf")
        bad[33, 3] = float("nan")
        z = ex.linear(bad, codes, su, sv, 2, scale, **kw)
        rest = torch.ones(T, dtype=torch.bool, device=DEV)
        rest[[5, 33]] = False
        assert torch.equal(z[rest], y[rest])
        assert not torch.isfinite(z[~rest]).any()


def test_gradients_of_small_sums_beside_large_ones(ex):
    """float16: an adapter's token with sums ten million times those of its others, and a
    gradient that is 0 in half of the columns: there the others are all there is."""
    g = gen(55)
    T = 90
    codes, su, sv, scale = coded(g, 256, 384, 2)
    x, dy = torch.randn(T, 256, generator=g, device=DEV) * 1e-3, torch.randn(T, 384, generator=g, device=DEV)
    x[4] *= 1e7
    dy[4, ::2] = 0
    x, dy = x.half(), dy.half()
    A = torch.randn(1, 6, 256, generator=g, device=DEV).half()
    B = (0.1 * torch.randn(1, 6, 384, generator=g, device=DEV)).half()
    slots = torch.zeros(T, dtype=torch.int32, device=DEV)
    got = ex.linear_backward(dy, x, codes, su, sv, 2, scale, A=A, B=B, gain=torch.ones(1, device=DEV), slots=slots)
    h = x.double() @ A[0].double().t()
    ref, e = h.t() @ dy.double(), (h.pow(2).t() @ dy.double().pow(2)).sqrt()
    tol = U["fp16"] * ref.abs() + 2.0 ** -25 + 6 * U["fp16"] / math.sqrt(3) * e
    live = torch.arange(384, device=DEV) % 2 == 0
    assert (ref[:, live].abs() < 10).all()
    assert ((got["dB"][0].double() - ref).abs() <= tol)[:, live].all()


@pytest.mark.parametrize("T", [3, 64, 65, 300])
def test_adapter_term_beyond_the_range_of_the_results(ex, T):
    """float16: the term alone is out of range where its sum with the coded part is not."""
    g = gen(52)
    codes, su, sv, scale = coded(g, 256, 384, 2)
    x = torch.randn(T, 256, generator=g, device=DEV).half()
    scale = scale * 3e4 / float((x.double() @ weight64(codes, su, sv, 2, scale)).std())
    W = weight64(codes, su, sv, 2, scale)
    base = x.double() @ W
    A = torch.randn(1, 1, 256, generator=g, device=DEV).half()
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    slots[1] = 0
    h = float(x[1].double() @ A[0, 0].double())
    B = (-2.5 * base[1] / h).half()[None, None]
    gain = torch.ones(1, device=DEV)
    term, err = adapter64(x, A, B, gain, slots, None)
    ref = base + term
    over = (term[1].abs() > 65520) & (ref[1].abs() < 65000)
    assert over.sum() > 10
    y = ex.linear(x, codes, su, sv, 2, scale, A=A, B=B, gain=gain, slots=slots)
    close(y[1:2, over], ref[1:2, over], sv.double()[over], "fp16", base[1:2, over], 6 * U["fp16"] / math.sqrt(3) * err[1:2, over])
    # the gradient of x is the same with the other transposition
    got = ex.linear_backward(x, torch.zeros(T, 384, dtype=torch.float16, device=DEV), codes.transpose(0, 1).contiguous(),
                             sv, su, 2, scale, A=B, B=A, gain=gain, slots=slots)["dx"]
    V = weight64(codes.transpose(0, 1).contiguous(), sv, su, 2, scale).t()
    base = x.double() @ V
    ref = base + term
    keep = ref.abs() < 65000
    assert torch.isfinite(got[keep]).all()


@pytest.mark.parametrize("T", [40, 64, 65, 700])
def test_adapter_term_that_cancels(ex, T):
    """bfloat16: the term takes most of the coded part away.  What stays has the rounding of
    the rotated activations (at most 2^-11 of each, 2^-11 / sqrt(3) as a root mean square; half
    as much again is allowed) and its own, not that of a term rounded before the sum."""
    g = gen(53)
    codes, su, sv, scale = coded(g, 512, 384, 4)
    W = weight64(codes, su, sv, 4, scale)
    x = torch.randn(T, 512, generator=g, device=DEV).bfloat16()
    base = x.double() @ W
    A = torch.randn(1, 1, 512, generator=g, device=DEV).bfloat16()
    for t in (0, T // 2, T - 1):
        slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
        slots[t] = 0
        h = float(x[t].double() @ A[0, 0].double())
        B = (-base[t] / h).bfloat16()[None, None]
        ref = base[t] + h * B[0, 0].double()
        y = ex.linear(x, codes, su, sv, 4, scale, A=A, B=B, gain=torch.ones(1, device=DEV), slots=slots)
        rms = lambda v: float(v.pow(2).mean().sqrt())  # noqa: E731
        assert rms(y[t].double() - ref) <= 1.5 * 2.0 ** -11 / math.sqrt(3) * rms(base[t]) + U["bf16"] * rms(ref)


@pytest.mark.parametrize("n", [256, 16512])
@pytest.mark.parametrize("T", [3, 70])
def test_row_scale_follows_the_products(ex, n, T):
    """A row's scale comes from its products with the channel factors: neither a value in a
    dead channel nor factors opposite to the activations take the rest's bits."""
    g = gen(54)
    codes, su, sv, scale = coded(g, 128, n, 2)
    sv = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, 1.0, -1.0)
    sv[7], sv[n - 1] = 0.0, 0.0
    x = torch.randn(T, n, generator=g, device=DEV)
    x[:, 7], x[:, n - 1] = 1e30, -1e25
    x = x.bfloat16()
    W = weight64(codes, su, sv, 2, scale).t()
    y = ex.linear(x, codes, su, sv, 2, scale, transposed=True)
    close(y, x.double() @ W, su.double(), "bf16")
    half = torch.arange(n, device=DEV) % 2 == 0
    f = torch.where(half, 2.0 ** 16, 2.0 ** -16)
    x = (torch.randn(T, n, generator=g, device=DEV) * f).bfloat16()
    sv = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, 1.0, -1.0) / f
    W = weight64(codes, su, sv, 2, scale).t()
    close(ex.linear(x, codes, su, sv, 2, scale, transposed=True), x.double() @ W, su.double(), "bf16")


@pytest.mark.parametrize("T", [3, 40, 70, 400])
def test_columns_of_one_buffer(ex, T):
    """Activations and results side by side in one buffer, as around a fused projection."""
    g = gen(56)
    codes, su, sv, scale = coded(g, 256, 384, 3)
    A, B, gain, ranks = adapters(g, 3, 8, 256, 384, "bf16")
    slots = torch.randint(-1, 3, (T,), generator=g, device=DEV, dtype=torch.int32)
    kw = dict(A=A, B=B, gain=gain, slots=slots, ranks=ranks)
    x, dy = acts(g, T, 256, "bf16"), acts(g, T, 384, "bf16")
    y, grad = ex.linear(x, codes, su, sv, 3, scale, **kw), ex.linear_backward(dy, x, codes, su, sv, 3, scale, **kw)
    buf = torch.full((T, 1408), 7.0, dtype=torch.bfloat16, device=DEV)
    bx, by, bd, bg = buf[:, 8:264], buf[:, 264:648], buf[:, 656:1040], buf[:, 1040:1296]
    bx.copy_(x), bd.copy_(dy)
    ex.linear(bx, codes, su, sv, 3, scale, out=by, **kw)
    got = ex.linear_backward(bd, bx, codes, su, sv, 3, scale, dx=bg, **kw)
    for p, q in ((bx, x), (by, y), (bd, dy), (bg, grad["dx"]), (got["dA"], grad["dA"]), (got["dB"], grad["dB"])):
        assert torch.equal(p, q)
    assert (buf[:, :8] == 7.0).all() and (buf[:, 648:656] == 7.0).all() and (buf[:, 1296:] == 7.0).all()
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    ex.expert_linear(bx, off, codes[None], su[None], sv[None], 3, scale[None], out=by)
    assert torch.equal(by, ex.expert_linear(x, off, codes[None], su[None], sv[None], 3, scale[None]))


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("T", [1, 40, 200])
def test_gradients_flow_through_the_calls(ex, T, tr):
    """x, A and B that want gradients get those of linear_backward, through whatever is
    around the call."""
    g = gen(57)
    codes, su, sv, scale = coded(g, 256, 384, 2)
    n_in, n_out = (384, 256) if tr else (256, 384)
    A, B, gain, ranks = adapters(g, 3, 8, n_in, n_out, "bf16")
    slots = torch.randint(-1, 3, (T,), generator=g, device=DEV, dtype=torch.int32)
    kw = dict(transposed=tr, gain=gain, slots=slots, ranks=ranks)
    x, c = acts(g, T, n_in, "bf16"), acts(g, T, n_out, "bf16")
    want = ex.linear_backward(c, x, codes, su, sv, 2, scale, A=A, B=B, **kw)
    plain = ex.linear(x, codes, su, sv, 2, scale, A=A, B=B, **kw)
    for wanted in ("x", "A", "B", "xAB"):
        t = dict(x=x.clone(), A=A.clone(), B=B.clone())
        for k in wanted:
            t[k].requires_grad_()
        y = ex.linear(t["x"], codes, su, sv, 2, scale, A=t["A"], B=t["B"], **kw)
        assert torch.equal(y, plain) and y.requires_grad
        y.backward(c)
        for k, v in t.items():
            assert (v.grad is not None) == (k in wanted)
            if k in wanted:
                assert torch.equal(v.grad, want["d" + k])
    # without adapters, and a gradient without strides of its own
    u = x.clone().requires_grad_()
    ex.linear(u, codes, su, sv, 2, scale, transposed=tr).sum().backward()
    ones = torch.ones(T, n_out, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(u.grad, ex.linear_backward(ones, None, codes, su, sv, 2, scale, transposed=tr)["dx"])
    with torch.no_grad():
        assert not ex.linear(u, codes, su, sv, 2, scale, transposed=tr).requires_grad
    # experts
    off = torch.tensor([0, T // 3, T // 3, max(T - 1, 1)], dtype=torch.int32, device=DEV)
    stack = [torch.stack([v] * 3) for v in (codes, su, sv)]
    scales = torch.stack([scale] * 3)
    u = x.clone().requires_grad_()
    z = ex.expert_linear(u, off, *stack, 2, scales, transposed=tr)
    z.backward(c)
    assert torch.equal(z, ex.expert_linear(x, off, *stack, 2, scales, transposed=tr))
    assert torch.equal(u.grad, ex.expert_linear(c, off, *stack, 2, scales, transposed=not tr))


# ---- forms that only large sizes reach ------------------------------------------------

@pytest.mark.parametrize("n", [16384, 16512, 28672])
@pytest.mark.parametrize("tr", [False, True])
def test_many_inputs(ex, n, tr):
    """Rows longer than one round of the rotation's block, aligned and not."""
    g = gen(n)
    rows, cols = (128, n) if tr else (n, 128)
    codes, su, sv, scale = coded(g, rows, cols, 2)
    W = weight64(codes, su, sv, 2, scale)
    W = W.t() if tr else W
    for T in (3, 70):
        for off in (8, 1):
            x = torch.full((T, n + 16), float("nan"), dtype=torch.bfloat16, device=DEV)[:, off:off + n]
            x.copy_(acts(g, T, n, "bf16"))
            close(ex.linear(x, codes, su, sv, 2, scale, transposed=tr), x.double() @ W, (su if tr else sv).double(), "bf16")


@pytest.mark.parametrize("K,dt,tr", [(1, "bf16", False), (4, "fp16", True), (2, "bf16", True), (3, "fp16", False)])
def test_pairs_with_two_accumulators(ex, K, dt, tr):
    """Tiles of more than 256 tokens, and more tiles than pairs of blocks."""
    g = gen(60 + K)
    codes, su, sv, scale = coded(g, 4096, 4096, K)
    W = weight64(codes, su, sv, K, scale)
    W = W.t() if tr else W
    A, B, gain, ranks = adapters(g, 3, 8, 4096, 4096, dt)
    for T in (333, 2100):
        x = acts(g, T, 4096, dt)
        slots = torch.randint(-1, 3, (T,), generator=g, device=DEV, dtype=torch.int32)
        y = ex.linear(x, codes, su, sv, K, scale, transposed=tr, A=A, B=B, gain=gain, slots=slots, ranks=ranks)
        term, err = adapter64(x, A, B, gain, slots, ranks)
        base = x.double() @ W
        close(y, base + term, (su if tr else sv).double(), dt, base, 6 * U[dt] / math.sqrt(3) * err)
        bad = x.clone()
        bad[1, 5], bad[T - 2, 9] = float("inf"), float("nan")
        z = ex.linear(bad, codes, su, sv, K, scale, transposed=tr, A=A, B=B, gain=gain, slots=slots, ranks=ranks)
        rest = torch.ones(T, dtype=torch.bool, device=DEV)
        rest[[1, T - 2]] = False
        assert torch.equal(z[rest], y[rest])
        assert not torch.isfinite(z[~rest][:, (su if tr else sv) != 0]).any()


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("tr", [False, True])
def test_blocks_with_several_tiles(ex, K, tr):
    """More tiles of 128 outputs than blocks: accumulators alternate, code rings go on."""
    g = gen(70 + K)
    rows, cols = (32768, 256) if tr else (256, 32768)
    codes, su, sv, scale = coded(g, rows, cols, K)
    W = weight64(codes, su, sv, K, scale)
    W = W.t() if tr else W
    for T in (65, 150, 256):
        x = acts(g, T, 256, "bf16")
        close(ex.linear(x, codes, su, sv, K, scale, transposed=tr), x.double() @ W, (su if tr else sv).double(), "bf16")


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("K,counts", [(2, [1100, 0, 700]), (3, [13, 1027, 1480]), (4, [2000]), (1, [600] * 9)])
def test_experts_in_pairs_and_many_tiles(ex, K, counts, tr):
    """More than 512 rows an expert on average: pairs of blocks; odd and empty groups,
    an odd number of output blocks."""
    g = gen(80 + K)
    E, rows, cols = len(counts), 384, 640
    codes, su, sv, scale = coded(g, rows, cols, K, (E,))
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    T = int(off[-1])
    x = acts(g, T, cols if tr else rows, "fp16")
    x[3, 1], x[T - 1, 2] = float("inf"), float("nan")
    y = ex.expert_linear(x, off, codes, su, sv, K, scale, transposed=tr)
    ok = torch.isfinite(x.float()).all(1)
    for e, m in enumerate(counts):
        if m:
            r = slice(int(off[e]), int(off[e + 1]))
            W = weight64(codes[e], su[e], sv[e], K, scale[e])
            right = (su if tr else sv)[e].double()
            close(y[r][ok[r]], x[r][ok[r]].double() @ (W.t() if tr else W), right, "fp16")
            assert not torch.isfinite(y[r][~ok[r]][:, right != 0]).any()


def test_experts_with_many_tiles_alone(ex):
    g = gen(90)
    E, rows, cols, K = 64, 128, 1024, 3
    codes, su, sv, scale = coded(g, rows, cols, K, (E,))
    p = torch.rand(E, generator=g, device=DEV) ** 3
    counts = torch.bincount(torch.multinomial(p, 1500, replacement=True, generator=g), minlength=E).tolist()
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    x = acts(g, 1500, rows, "bf16")
    y = ex.expert_linear(x, off, codes, su, sv, K, scale)
    for e, m in enumerate(counts):
        r = slice(int(off[e]), int(off[e + 1]))
        if m:
            close(y[r], x[r].double() @ weight64(codes[e], su[e], sv[e], K, scale[e]), sv[e].double(), "bf16")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,n", [(4097, 3), (9001, 40)])
def test_adapters_of_more_tokens_than_a_round_of_the_plan(ex, dt, T, n):
    g = gen(T)
    codes, su, sv, scale = coded(g, 128, 256, 2)
    W = weight64(codes, su, sv, 2, scale)
    A, B, gain, ranks = adapters(g, n, 8, 128, 256, dt)
    slots = torch.randint(-1, n, (T,), generator=g, device=DEV, dtype=torch.int32)
    x, dy = acts(g, T, 128, dt), acts(g, T, 256, dt, 0.1)
    kw = dict(A=A, B=B, gain=gain, slots=slots, ranks=ranks)
    y = ex.linear(x, codes, su, sv, 2, scale, **kw)
    term, err = adapter64(x, A, B, gain, slots, ranks)
    base = x.double() @ W
    close(y, base + term, sv.double(), dt, base, 6 * U[dt] / math.sqrt(3) * err)
    got = ex.linear_backward(dy, x, codes, su, sv, 2, scale, **kw)
    term, err = adapter64(dy, B, A, gain, slots, ranks)
    base = dy.double() @ W.t()
    close(got["dx"], base + term, su.double(), dt, base, 6 * U[dt] / math.sqrt(3) * err)
    for i in range(n):
        t, k = torch.nonzero(slots == i).flatten(), int(ranks[i])
        X, D = x[t].double(), dy[t].double()
        gg, h = float(gain[i]) * (D @ B[i, :k].double().t()), float(gain[i]) * (X @ A[i, :k].double().t())
        for name, p, q in (("dA", gg, X), ("dB", h, D)):
            ref, e = p.t() @ q, (p.pow(2).t() @ q.pow(2)).sqrt()
            tol = U[dt] * ref.abs() + 2.0 ** -25 + 6 * U[dt] / math.sqrt(3) * e
            assert ((got[name][i, :k].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_rows_that_are_not_numbers_stay_alone(ex, dt):
    """With adapters, in gradients and in few-row experts."""
    g = gen(91)
    codes, su, sv, scale = coded(g, 256, 384, 3)
    for T in (4, 33, 64, 90):
        A, B, gain, ranks = adapters(g, 2, 8, 256, 384, dt)
        slots = (torch.arange(T, device=DEV) % 3 - 1).int()
        x, dy = acts(g, T, 256, dt), acts(g, T, 384, dt)
        bad, dbad = x.clone(), dy.clone()
        bad[1, 7], bad[T - 1, 130] = float("-inf"), float("nan")
        dbad[1, 7], dbad[T - 1, 130] = float("nan"), float("inf")
        rest = torch.ones(T, dtype=torch.bool, device=DEV)
        rest[[1, T - 1]] = False
        kw = dict(A=A, B=B, gain=gain, slots=slots, ranks=ranks)
        y, z = (ex.linear(v, codes, su, sv, 3, scale, **kw) for v in (x, bad))
        assert torch.equal(y[rest], z[rest]) and not torch.isfinite(z[~rest][:, sv != 0]).any()
        y, z = (ex.linear_backward(v, x, codes, su, sv, 3, scale, **kw)["dx"] for v in (dy, dbad))
        assert torch.equal(y[rest], z[rest]) and not torch.isfinite(z[~rest]).any()
        off = torch.tensor([0, 2, 2, T - 1, T], dtype=torch.int32, device=DEV)
        stack = [torch.stack([v] * 4) for v in (codes, su, sv)]
        y, z = (ex.expert_linear(v, off, *stack, 3, torch.stack([scale] * 4)) for v in (x, bad))
        assert torch.equal(y[rest], z[rest]) and not torch.isfinite(z[~rest][:, sv != 0]).any()
