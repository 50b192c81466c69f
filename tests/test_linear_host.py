"""Refusals of the products with coded matrices (not gpu): arguments are checked
before anything reaches the GPU, so fake pointers are never dereferenced."""
import ctypes

import pytest

FAKE = 0x10000000
Y = 0x20000000
WS = 0x40000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def ex():
    from exl3_trellis_weight_gb300 import build
    build.build()
    import exl3_trellis_weight_gb300 as ex
    ex.lib()
    return ex


def _linear(ex, **kw):
    a = dict(x=FAKE, dt=1, T=4, xs=256, codes=FAKE, rows=256, cols=384, K=2, su=FAKE, sv=FAKE, scale=FAKE, tr=0,
             A=FAKE, B=FAKE, gain=FAKE, slots=FAKE, ranks=None, n=2, r=8, y=Y, ys=384, ws=WS, wb=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return ex.lib().exl3_linear(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dt=0)), (1, dict(dt=3)), (1, dict(T=-1)), (1, dict(T=(1 << 24) + 1)),
    (2, dict(rows=200)), (2, dict(cols=64)), (2, dict(rows=0)), (2, dict(rows=1 << 17)), (2, dict(K=0)), (2, dict(K=5)),
    (1, dict(codes=None)), (1, dict(codes=FAKE + 4)), (1, dict(su=None)), (1, dict(su=FAKE + 4)),
    (1, dict(sv=None)), (1, dict(scale=None)), (1, dict(scale=FAKE + 2)),
    (1, dict(x=None)), (1, dict(x=FAKE + 1)), (1, dict(xs=255)), (1, dict(xs=-256)), (1, dict(y=None)),
    (1, dict(ys=383)), (1, dict(y=FAKE)), (1, dict(y=FAKE + 2 * (3 * 256 + 255))), (1, dict(y=FAKE - 2 * (3 * 384 + 383))),
    (2, dict(n=-1)), (2, dict(n=1025)), (2, dict(r=0)), (2, dict(r=129)),
    (1, dict(A=None)), (1, dict(B=None)), (1, dict(B=FAKE + 8)), (1, dict(gain=None)), (1, dict(slots=None)),
    (1, dict(ranks=FAKE + 2)),
    (1, dict(ws=None)), (1, dict(ws=WS + 16)), (3, dict(wb=1024)), (1, dict(ws=Y - 256)),
])
def test_linear_refuses(ex, want, kw):
    assert _linear(ex, **kw) == want
    assert ex.lib().exl3_last_error()


def test_linear_with_no_tokens_does_nothing(ex):
    assert _linear(ex, T=0, x=None, y=None, slots=None, ws=None, wb=0) == 0


def test_workspace_is_as_large_as_the_query_says(ex):
    need = ex.linear_workspace_bytes(4, 256, 384, False, 2, 8)
    assert need > 0 and _linear(ex, wb=need - 1) == 3
    assert ex.linear_workspace_bytes(4, 200, 384) == 0
    assert ex.linear_workspace_bytes(-1, 256, 384) == 0
    assert ex.linear_workspace_bytes(4, 256, 384, False, 2, 200) == 0
    assert ex.linear_backward_workspace_bytes(4, 256, 384, False, 2, 8) > 0
    assert ex.linear_backward_workspace_bytes(4, 256, 100) == 0
    assert ex.expert_linear_workspace_bytes(4, 256, 384) > 0
    assert ex.expert_linear_workspace_bytes(4, 256, 0) == 0
    # the rotated activations: two bytes for each
    assert ex.linear_workspace_bytes(4096, 4096, 128) >= 4096 * 4096 * 2


def _backward(ex, **kw):
    a = dict(dy=FAKE, dys=384, x=0x18000000, xs=256, dt=2, T=4, codes=FAKE, rows=256, cols=384, K=3, su=FAKE, sv=FAKE,
             scale=FAKE, tr=0, A=FAKE, B=FAKE, gain=FAKE, slots=FAKE, ranks=None, n=2, r=8, dx=Y, dxs=256,
             dA=0x30000000, dB=0x38000000, ws=WS, wb=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return ex.lib().exl3_linear_backward(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dt=0)), (2, dict(rows=64)), (2, dict(K=9)), (1, dict(dy=None)), (1, dict(dys=256)), (1, dict(x=None)),
    (1, dict(xs=100)), (1, dict(dx=None)), (1, dict(dxs=255)), (1, dict(dA=None)), (1, dict(dB=None)),
    (1, dict(dA=0x30000002)), (1, dict(dx=FAKE)), (1, dict(dx=0x18000000)), (2, dict(n=2000)), (2, dict(r=1000)),
    (1, dict(ws=None)), (3, dict(wb=100)), (1, dict(slots=None)),
])
def test_backward_refuses(ex, want, kw):
    assert _backward(ex, **kw) == want


def test_backward_of_nothing_does_nothing(ex):
    assert _backward(ex, T=0, n=0, r=0, dy=None, x=None, dx=None, A=None, B=None, gain=None, slots=None, dA=None,
                     dB=None, ws=None, wb=0) == 0


def _experts(ex, **kw):
    a = dict(x=FAKE, dt=1, T=4, xs=256, off=FAKE, E=3, codes=FAKE, rows=256, cols=384, K=2, su=FAKE, sv=FAKE,
             scale=FAKE, tr=0, y=Y, ys=384, ws=WS, wb=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return ex.lib().exl3_expert_linear(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dt=0)), (1, dict(T=-1)), (2, dict(E=0)), (2, dict(E=1025)), (1, dict(off=None)), (1, dict(off=FAKE + 2)),
    (2, dict(rows=130)), (2, dict(K=6)), (1, dict(x=None)), (1, dict(ys=100)), (1, dict(tr=1, xs=256, ys=256)),
    (1, dict(y=FAKE)), (1, dict(ws=WS + 1)), (3, dict(wb=0)),
])
def test_experts_refuse(ex, want, kw):
    assert _experts(ex, **kw) == want


def test_python_checks_need_no_gpu(ex):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    codes = torch.zeros(16, 8, 32, dtype=torch.int16)
    su, sv, s = torch.zeros(256), torch.zeros(128), torch.ones(())
    with pytest.raises(ValueError, match="CUDA"):
        ex.linear(x, codes, su, sv, 2, s)
    with pytest.raises(ValueError, match="codes must be"):
        ex.linear(x, codes, su, sv, 4, s)
    with pytest.raises(ValueError, match="dimensions"):
        ex.linear(x, codes[0], su, sv, 2, s)
    with pytest.raises(ValueError, match="int16"):
        ex.linear(x, codes.int(), su, sv, 2, s)
    with pytest.raises(ValueError, match="codes must be"):
        ex.linear(x, codes, su, sv, 3, s)
    with pytest.raises(ValueError, match="su must be"):
        ex.linear(x, codes, sv, sv, 2, s)
    with pytest.raises(ValueError, match="contiguous"):
        ex.linear(x, codes, su.repeat(2)[::2], sv, 2, s)
    with pytest.raises(ValueError, match="experts"):
        ex.expert_linear(x, torch.zeros(2, dtype=torch.int32), codes, su, sv, 2, s)
    with pytest.raises(AttributeError):
        ex.no_such_entry_point
    assert ctypes.sizeof(ctypes.c_void_p) == 8
