"""What the calls around the coded products take for granted of torch, and their outputs under
autograd, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_layer import DEV, acts, gen  # noqa: E402


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


@pytest.mark.parametrize("shape,stride", [((3, 5), (5, 1)), ((7, 4), (1, 7)), ((0, 8), (8, 1)), ((0, 4), (1, 0)), ((256,), (1,))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.uint8])
def test_allocations_are_torchs(ex, shape, stride, dtype):
    """The short way to an allocation, a private name of torch's, gives what torch.empty_strided does,
    from the stream's own part of the caching allocator."""
    from exl3_trellis_weight_gb300 import layer
    for make in (layer._maker(0), lambda *a: layer._maker(0)(*a)):
        t, u = make(shape, stride, dtype), torch.empty_strided(shape, stride, dtype=dtype, device=DEV)
        assert (t.shape, t.stride(), t.dtype, t.device, t.storage_offset()) == (u.shape, u.stride(), u.dtype, u.device, u.storage_offset())
        assert t.untyped_storage().nbytes() == u.untyped_storage().nbytes()
        assert type(t) is torch.Tensor and not t.requires_grad and not t.is_inference() and t.is_leaf
    del t, u
    held = torch.cuda.memory_allocated()
    t = layer._maker(0)((1 << 20,), (1,), torch.uint8)
    assert torch.cuda.memory_allocated() == held + (1 << 20)
    del t
    assert torch.cuda.memory_allocated() == held
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):          # a block of another stream is not handed out on this one
        a = layer._maker(0)((1 << 20,), (1,), torch.uint8).data_ptr()
    b = layer._maker(0)((1 << 20,), (1,), torch.uint8).data_ptr()
    assert a != b


def test_a_saved_residual_that_is_overwritten(ex):
    g = gen(1)
    x, r, w = acts(g, 9, 512, "bf16"), acts(g, 9, 512, "bf16"), torch.rand(512, generator=g, device=DEV)
    leaf = torch.ones_like(r).requires_grad_()
    loss = (leaf * r).sum()
    want = ex.rms_norm(x, w, residual=r)["h"]
    got = ex.rms_norm(x, w, residual=r, h=r)["h"]
    assert got is r and torch.equal(r, want)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        t = r.clone()
        ex.rms_norm(x, w, residual=t, h=t, out=x.clone())
