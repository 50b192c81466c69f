"""Gradients of norms with many rows to a block: the ring of whole rows goes around (its stages are
asked for again, the phases of its barriers turn), with two and three operands to a stage."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_layer import DEV, acts, gen, test_norm_gradient as check_gradient  # noqa: E402

# rows, columns, rows that all blocks take at a time (152 SMs), stages: T is twice their product at least
SIZES = [(30011, 512, 2432, 6), (26003, 520, 1520, 8), (15001, 1024, 1216, 6), (8001, 2048, 608, 6), (4001, 4096, 304, 6), (2000, 8192, 152, 6)]


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


def test_the_ring_goes_around():
    assert all(T >= 2 * at_once * depth for T, _, at_once, depth in SIZES)


@pytest.mark.parametrize("T,n", [s[:2] for s in SIZES])
@pytest.mark.parametrize("dt,w32", [("bf16", True), ("fp16", False), ("bf16", False)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_many_rows_a_block(ex, T, n, dt, w32, with_dh):
    check_gradient(ex, T, n, dt, with_dh, False, w32)
    if with_dh:                            # dx over dy, beside dh
        g = gen(n)
        h, dy, dh = acts(g, T, n, dt), acts(g, T, n, dt, scale=0.1), acts(g, T, n, dt, scale=0.1)
        w = torch.rand(n, generator=g, device=DEV) + 0.5
        want = ex.rms_norm_backward(dy, h, w, dh=dh)
        got = ex.rms_norm_backward(dy, h, w, dh=dh, dx=dy)
        assert got["dx"] is dy and torch.equal(dy, want["dx"]) and torch.equal(got["dweight"], want["dweight"])
