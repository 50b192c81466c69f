"""Workspaces and arguments of the products with coded matrices (not gpu): nothing here
reaches the GPU, fake pointers are never dereferenced."""
import pytest


@pytest.fixture(scope="module")
def ex():
    from exl3_trellis_weight_gb300 import build
    build.build()
    import exl3_trellis_weight_gb300 as ex
    ex.lib()
    return ex


@pytest.mark.parametrize("T", [0, 1, 64, 65, 700, 4096])
@pytest.mark.parametrize("rows,cols", [(512, 1024), (1024, 512), (128, 65536)])
@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("n,r", [(0, 0), (1, 1), (5, 48)])
def test_a_workspace_for_the_gradients_serves_the_product(ex, T, rows, cols, tr, n, r):
    grad, product = (f(T, rows, cols, tr, n, r) for f in (ex.linear_backward_workspace_bytes, ex.linear_workspace_bytes))
    assert grad >= product > 0


# addresses far apart for every argument, each array within its 16 MB
CODES, SU, SV, SCALE, X, DY, A, B, GAIN, SLOTS, Y, DA, DB, WS = (0x10000000 + 0x1000000 * i for i in range(14))
T, ROWS, COLS, N, R = 4, 256, 384, 2, 8


def _linear(ex, **kw):
    a = dict(x=X, dt=1, T=T, xs=ROWS, codes=CODES, rows=ROWS, cols=COLS, K=2, su=SU, sv=SV, scale=SCALE, tr=0, A=A, B=B,
             gain=GAIN, slots=SLOTS, ranks=None, n=N, r=R, y=Y, ys=COLS, ws=WS, wb=0)
    a.update(kw)
    return ex.lib().exl3_linear(*a.values(), None)


def _backward(ex, **kw):
    a = dict(dy=DY, dys=COLS, x=X, xs=ROWS, dt=2, T=T, codes=CODES, rows=ROWS, cols=COLS, K=3, su=SU, sv=SV, scale=SCALE,
             tr=0, A=A, B=B, gain=GAIN, slots=SLOTS, ranks=None, n=N, r=R, dx=Y, dxs=ROWS, dA=DA, dB=DB, ws=WS, wb=1 << 20)
    a.update(kw)
    return ex.lib().exl3_linear_backward(*a.values(), None)


SIZE_A, SIZE_B = 2 * N * R * ROWS, 2 * N * R * COLS


@pytest.mark.parametrize("kw", [
    # the gradients of A and B start while the product still reads, and write while x and dy are read
    dict(dA=A), dict(dA=A + SIZE_A - 16), dict(dB=A + 16), dict(dA=B), dict(dB=B), dict(dB=B - SIZE_B + 16),
    dict(dA=X), dict(dA=X + 2 * T * ROWS - 16), dict(dB=X), dict(dA=DY), dict(dB=DY + 16), dict(dA=CODES), dict(dB=CODES + 16),
    dict(dA=Y), dict(dB=Y + 2 * T * ROWS - 16), dict(dA=WS), dict(dB=WS + 4096), dict(dA=DB), dict(dB=DA + SIZE_A - 16),
    dict(dx=A + 2), dict(dx=B), dict(dx=CODES),
])
def test_gradients_refuse_outputs_over_what_they_read(ex, kw):
    assert _backward(ex, **kw) == 1
    assert b"overlaps" in ex.lib().exl3_last_error()


def test_gradients_take_neighbouring_outputs(ex):
    for kw in (dict(), dict(dA=A + SIZE_A, dB=B - SIZE_B), dict(dB=DA + SIZE_A), dict(dA=X + 2 * T * ROWS)):
        assert _backward(ex, wb=0, **kw) == 3


@pytest.mark.parametrize("kw", [dict(y=A), dict(y=B + SIZE_B - 2), dict(y=CODES + ROWS * COLS // 4 - 2)])
def test_products_refuse_results_over_what_they_read(ex, kw):
    assert _linear(ex, **kw) == 1
    assert b"overlaps" in ex.lib().exl3_last_error()


def test_experts_refuse_results_over_the_codes(ex):
    E, size = 3, ROWS * COLS * 2 // 8
    for y, want in ((CODES, 1), (CODES + E * size - 2, 1), (CODES + E * size, 3)):
        assert ex.lib().exl3_expert_linear(X, 1, T, ROWS, SLOTS, E, CODES, ROWS, COLS, 2, SU, SV, SCALE, 0, y, COLS, WS, 0,
                                           None) == want


@pytest.mark.parametrize("at,want", [
    # y's columns in a buffer whose rows of 1024 begin with x's 256: beside them, up to their end,
    # touching their last or (a row on) their first element
    (256, 3), (640, 3), (255, 1), (641, 1), (0, 1), (-384, 3), (-385, 3), (-383, 1), (1024 + 256, 3), (1024 + 255, 1),
])
def test_columns_of_one_buffer_may_stand_side_by_side(ex, at, want):
    assert _linear(ex, xs=1024, ys=1024, y=X + 2 * at, n=0) == want
    assert ex.lib().exl3_expert_linear(X, 1, T, 1024, SLOTS, 1, CODES, ROWS, COLS, 2, SU, SV, SCALE, 0, X + 2 * at, 1024,
                                       WS, 0, None) == want


def test_columns_of_different_strides_are_compared_whole(ex):
    assert _linear(ex, xs=1024, ys=1032, y=X + 2 * 256, n=0) == 1
    assert _linear(ex, xs=1024, ys=1032, y=X + 2 * (3 * 1024 + 256), n=0) == 3
    # a single row has no stride
    assert _linear(ex, T=1, xs=256, ys=384, y=X + 2 * 256, n=0) == 3
    assert _linear(ex, T=1, xs=256, ys=384, y=X + 2 * 255, n=0) == 1
    assert _linear(ex, T=1, xs=300, ys=300 + 84, y=X + 2 * 128, n=0) == 1


def test_gradient_beside_its_input(ex):
    # dx (256 columns) behind dy's 384 and x's 256 in rows of 1024
    def at(dx, x):
        return _backward(ex, dys=1024, xs=1024, dxs=1024, x=DY + 2 * x, dx=DY + 2 * dx, wb=0)
    assert at(640, 384) == 3 and at(768, 384) == 3
    assert at(639, 384) == 1 and at(383, 640) == 1 and at(769, 384) == 1
