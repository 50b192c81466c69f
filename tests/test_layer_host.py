"""Refusals of norms, 8-bit blocks and products and whole expert layers (not gpu): arguments
are checked before anything reaches the GPU, so fake pointers are never dereferenced."""
import ctypes
import math

import pytest

# addresses far apart, each array within its 16 MB
X, R, W, H, Y, Q, S, DY, DH, DX, DW, WS, C, SU, SV, SC, IDS, PW, RT = (0x10000000 + 0x1000000 * i for i in range(19))
BIG = 1 << 40
F32, BF16, F16, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def ex():
    from exl3_trellis_weight_gb300 import build
    build.build()
    import exl3_trellis_weight_gb300 as ex
    ex.lib()
    return ex


def _norm(ex, **kw):
    a = dict(x=X, dt=BF16, T=4, n=256, xs=256, r=R, rs=256, w=W, wdt=BF16, eps=1e-6, h=H, hs=256, y=Y, ys=256, y8=Q, scale=S)
    assert set(kw) <= set(a)
    a.update(kw)
    return ex.lib().exl3_rms_norm(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dt=F32)), (1, dict(dt=E4M3)), (1, dict(T=-1)), (1, dict(T=(1 << 24) + 1)), (2, dict(n=0)), (2, dict(n=32769)),
    (1, dict(w=None)), (1, dict(w=W + 1)), (1, dict(wdt=F16)), (1, dict(wdt=F32, w=W + 2)),
    (1, dict(eps=0.0)), (1, dict(eps=-1e-6)), (1, dict(eps=math.nan)), (1, dict(eps=math.inf)), (1, dict(eps=1e-40)),
    (1, dict(x=None)), (1, dict(x=X + 1)), (1, dict(xs=255)), (1, dict(rs=100)), (1, dict(h=None)), (1, dict(hs=255)),
    (1, dict(y=None, y8=None, scale=None)), (1, dict(y8=None)), (1, dict(scale=None)), (1, dict(scale=S + 2)),
    # outputs over inputs or each other
    (1, dict(h=X + 2)), (1, dict(h=X, hs=512)), (1, dict(h=R - 2)), (1, dict(h=W)), (1, dict(y=R)), (1, dict(y=H)), (1, dict(y=X + 512)),
    (1, dict(y=X, ys=300)), (1, dict(y=W)), (1, dict(y8=X)), (1, dict(y8=R + 16)), (1, dict(y8=H)), (1, dict(y8=Y + 8)), (1, dict(y8=W)),
    (1, dict(scale=X)), (1, dict(scale=Y)), (1, dict(scale=Q)), (1, dict(y8=S - 1023)),
])
def test_norm_refuses(ex, want, kw):
    assert _norm(ex, **kw) == want
    assert ex.lib().exl3_last_error()


def test_norm_of_nothing(ex):
    assert _norm(ex, T=0, x=None, r=None, h=None, y=None, y8=None, scale=None) == 0


def _grad(ex, **kw):
    a = dict(dy=DY, gs=256, h=H, hs=256, dt=F16, T=4, n=256, w=W, wdt=F32, eps=1e-6, dh=DH, ds=256, dx=DX, xs=256, dw=DW, ws=WS, wb=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return ex.lib().exl3_rms_norm_backward(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dt=F32)), (2, dict(n=40000)), (1, dict(wdt=BF16)), (1, dict(w=None)), (1, dict(eps=0.0)), (1, dict(dy=None)), (1, dict(gs=1)),
    (1, dict(h=None)), (1, dict(hs=255)), (1, dict(dh=DH + 1)), (1, dict(ds=0)), (1, dict(dx=None)), (1, dict(xs=255)),
    (1, dict(dx=H)), (1, dict(dx=DY + 2)), (1, dict(dx=DY, xs=257)), (1, dict(dx=DH + 512)), (1, dict(dx=W)), (1, dict(dx=WS, wb=BIG)),
    (1, dict(dw=DW + 2)), (1, dict(dw=DY)), (1, dict(dw=H)), (1, dict(dw=DH)), (1, dict(dw=DX)), (1, dict(dw=W)), (1, dict(dw=WS + 256, wb=BIG)),
    (1, dict(ws=None)), (1, dict(ws=WS + 8)), (3, dict()),
])
def test_norm_gradient_refuses(ex, want, kw):
    assert _grad(ex, **kw) == want


def test_norm_gradient_takes_dy_or_dh_for_dx(ex):
    for kw in (dict(), dict(dx=DY), dict(dx=DH), dict(dw=DW, dh=None, ds=0)):
        assert _grad(ex, **kw) == 3        # all but the workspace is right
    need = ex.rms_norm_backward_workspace_bytes(4, 256)
    assert need > 0 and _grad(ex, wb=need - 1) == 3
    assert ex.rms_norm_backward_workspace_bytes(4, 0) == 0 and ex.rms_norm_backward_workspace_bytes(-1, 64) == 0
    assert ex.rms_norm_backward_workspace_bytes(0, 64) > 0


def _q8(ex, **kw):
    a = dict(x=X, dt=F32, T=130, n=256, xs=256, rows=128, codes=Q, scale=S)
    assert set(kw) <= set(a)
    a.update(kw)
    return ex.lib().exl3_quantize8(*a.values(), None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dt=E4M3)), (1, dict(T=-1)), (1, dict(T=(1 << 24) + 1)), (2, dict(n=0)), (2, dict(n=65537)), (2, dict(rows=2)), (2, dict(rows=0)),
    (1, dict(x=None)), (1, dict(x=X + 2)), (1, dict(xs=255)), (1, dict(codes=None)), (1, dict(scale=None)), (1, dict(scale=S + 1)),
    (1, dict(codes=X)), (1, dict(codes=X + 130 * 256 * 4 - 1)), (1, dict(scale=X + 4)), (1, dict(scale=Q)), (1, dict(codes=S, rows=1)),
])
def test_blocks_refuse(ex, want, kw):
    assert _q8(ex, **kw) == want


def _lin(ex, **kw):
    a = dict(x=X, dt=BF16, T=4, xs=256, s=None, st=0, sb=0, w=C, ws=SC, rows=256, cols=384, tr=0, y=Y, ydt=BF16, ys=384, wk=WS, wb=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return ex.lib().exl3_linear8(*a.values(), None)


CODED = dict(dt=E4M3, s=S, st=1, sb=4)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dt=F32)), (1, dict(ydt=F32)), (1, dict(ydt=E4M3)), (1, dict(T=-1)), (2, dict(rows=250)), (2, dict(cols=8)), (2, dict(rows=1 << 17)),
    (2, dict(cols=0)), (1, dict(w=None)), (1, dict(w=C + 8)), (1, dict(ws=None)), (1, dict(ws=SC + 2)), (1, dict(x=None)), (1, dict(x=X + 1)),
    (1, dict(xs=255)), (1, dict(y=None)), (1, dict(ys=383)), (1, dict(tr=1, xs=256)), (1, dict(y=X)), (1, dict(y=C)), (1, dict(y=SC)),
    (1, dict(s=S)), (1, dict(wk=None)), (1, dict(wk=WS + 16)), (3, dict()), (1, dict(y=WS, wb=BIG)),
    (1, dict(CODED, x=X + 8)), (1, dict(CODED, xs=264)), (1, dict(CODED, s=None)), (1, dict(CODED, s=S + 2)), (1, dict(CODED, st=-1)),
    (1, dict(CODED, sb=-4)), (1, dict(CODED, st=(1 << 32) + 1)), (1, dict(CODED, y=S)), (1, dict(CODED, y=X)),
])
def test_product_refuses(ex, want, kw):
    assert _lin(ex, **kw) == want


def test_product_workspace(ex):
    need = ex.linear8_workspace_bytes(4, 256, 384)
    assert need >= 4 * 256 + 4 * 2 * 4 and _lin(ex, wb=need - 1) == 3
    assert ex.linear8_workspace_bytes(4, 256, 384, True) >= 4 * 384
    assert ex.linear8_workspace_bytes(4, 100, 384) == 0 and ex.linear8_workspace_bytes(-1, 256, 384) == 0
    assert _lin(ex, T=0, x=None, y=None, wk=None) == 0


class Coded(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("su", ctypes.c_void_p), ("sv", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


def _experts(ex, at=None, **kw):
    """`at`: (matrix, field, address) of one pointer to change."""
    m = (Coded * 3)(*(Coded(C + i * 0x10000000, SU + i * 0x10000000, SV + i * 0x10000000, SC + i * 0x10000000) for i in range(3)))
    if at:
        setattr(m[at[0]], at[1], at[2])
    a = dict(x=X, dt=BF16, T=4, xs=256, router=RT, rdt=BF16, ids=None, weights=None, top_k=2, norm=1, E=5, experts=ctypes.cast(m, ctypes.c_void_p),
             H=256, F=384, K=2, Kd=3, tr=0, y=Y, ys=256, ws=WS, wb=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return ex.lib().exl3_expert_layer(*a.values(), None)


GIVEN = dict(router=None, ids=IDS, weights=PW)


@pytest.mark.parametrize("want,kw", [
    (1, dict(dt=F32)), (1, dict(dt=E4M3)), (2, dict(E=0)), (2, dict(E=1025)), (2, dict(top_k=0)), (2, dict(top_k=6)), (2, dict(top_k=33, E=64)),
    (2, dict(T=-1)), (2, dict(T=257)), (2, dict(T=200, top_k=21, E=64)), (2, dict(H=200)), (2, dict(F=64)), (2, dict(H=0)), (2, dict(F=32896)),
    (2, dict(K=0)), (2, dict(K=5)), (2, dict(Kd=9)), (1, dict(experts=None)),
    (1, dict(at=(0, "codes", None))), (1, dict(at=(1, "codes", C + 8))), (1, dict(at=(2, "su", None))), (1, dict(at=(0, "sv", SV + 4))),
    (1, dict(at=(1, "scale", None))), (1, dict(at=(2, "scale", SC + 2))),
    (1, dict(rdt=F16)), (1, dict(rdt=F32, router=RT + 2)), (1, dict(ids=IDS)), (1, dict(weights=PW)), (1, dict(router=None)),
    (1, dict(GIVEN, ids=None)), (1, dict(GIVEN, weights=None)), (1, dict(GIVEN, ids=IDS + 2)), (1, dict(GIVEN, weights=PW + 1)),
    (1, dict(x=None)), (1, dict(xs=255)), (1, dict(y=None)), (1, dict(ys=255)), (1, dict(y=X)), (1, dict(y=RT)), (1, dict(y=C)),
    (1, dict(y=SU + 0x10000000)), (1, dict(y=SV + 0x20000000)), (1, dict(y=SC)), (1, dict(GIVEN, y=IDS)), (1, dict(GIVEN, y=PW)),
    (1, dict(ws=None)), (1, dict(ws=WS + 64)), (3, dict()), (3, GIVEN), (1, dict(y=WS + 512, wb=BIG)),
])
def test_expert_layer_refuses(ex, want, kw):
    assert _experts(ex, **kw) == want
    assert ex.lib().exl3_last_error()


def test_expert_layer_workspace(ex):
    need = ex.expert_layer_workspace_bytes(4, 256, 384, 5, 2)
    assert need > 0 and _experts(ex, wb=need - 1) == 3
    for bad in ((4, 200, 384, 5, 2), (4, 256, 0, 5, 2), (257, 256, 384, 5, 2), (4, 256, 384, 5, 6), (4, 256, 384, 2000, 2), (-1, 256, 384, 5, 2)):
        assert ex.expert_layer_workspace_bytes(*bad) == 0
    assert _experts(ex, T=0, x=None, y=None, ws=None) == 0
    # it does not shrink as tokens come, so one for the most serves them all
    sizes = [ex.expert_layer_workspace_bytes(T, 256, 384, 64, 8) for T in range(1, 257)]
    assert sizes == sorted(sizes)


def test_python_checks_need_no_gpu(ex):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    w = torch.ones(256)
    with pytest.raises(ValueError, match="CUDA"):
        ex.rms_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ex.rms_norm_backward(x, x, w)
    with pytest.raises(ValueError, match="CUDA"):
        ex.quantize8(x)
    with pytest.raises(ValueError, match="float8"):
        ex.linear8(x, x, w)
    codes = torch.zeros(3, 16, 8, 32, dtype=torch.int16)
    m = (codes, torch.zeros(3, 256), torch.zeros(3, 128), torch.ones(3))
    down = (codes.transpose(1, 2).contiguous(), m[2], m[1], m[3])
    with pytest.raises(ValueError, match="go together"):
        ex.expert_layer(x, m, m, m, 2, 1, router=x)
    with pytest.raises(ValueError, match="gate codes"):
        ex.expert_layer(x, m, m, down, 3, 1, router=x)
    with pytest.raises(ValueError, match="up su"):
        ex.expert_layer(x, m, (codes, m[2], m[2], m[3]), down, 2, 1, router=x)
    with pytest.raises(ValueError, match="CUDA"):
        ex.expert_layer(x, m, m, down, 2, 1, router=x)
