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
