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


def test_a_tensor_that_is_its_own_residual(ex):
    g = gen(2)
    x, w, dy = acts(g, 70, 640, "bf16"), torch.rand(640, generator=g, device=DEV), acts(g, 70, 640, "bf16", scale=0.1)
    h = (2 * x.float()).bfloat16()
    want, dx = ex.rms_norm(h, w)["y"], ex.rms_norm_backward(dy, h, w)["dx"]
    leaf, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
    r = ex.rms_norm(leaf, wl, residual=leaf)
    assert torch.equal(r["h"], h) and torch.equal(r["y"], want)
    r["y"].backward(dy)
    assert torch.equal(leaf.grad, (2 * dx.float()).bfloat16())
    # and updated where it lies
    t = x.clone()
    got = ex.rms_norm(t, w, residual=t, h=t)
    assert torch.equal(t, h) and torch.equal(got["y"], want)


def test_gradients_without_tokens(ex):
    x, w = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV).requires_grad_(), torch.ones(256, device=DEV).requires_grad_()
    q, s = ex.quantize8(torch.randn(256, 128, device=DEV), block_rows=128)
    ex.linear8(ex.rms_norm(x, w)["y"], q, s).sum().backward()
    assert x.grad.shape == (0, 256) and bool((w.grad == 0).all())


@pytest.mark.parametrize("T", [1, 20, 64, 100, 400])
@pytest.mark.parametrize("tr", [False, True])
def test_8_bit_rows_and_scales_of_wider_buffers(ex, T, tr):
    """Rows of x 16 bytes into a wider buffer, scales by token, by block, every other one, and one for
    all tokens."""
    g = gen(T)
    n, n_out = 656, 272
    w, ws = ex.quantize8(torch.randn(*((n_out, n) if tr else (n, n_out)), generator=g, device=DEV), block_rows=128)
    codes, scale = ex.quantize8(acts(g, T, n, "bf16"))
    want = ex.linear8(codes, w, ws, scale, transposed=tr)
    buf = torch.full((T, n + 64), 0x7F, dtype=torch.uint8, device=DEV)         # (NaN beside the rows)
    buf[:, 16:16 + n] = codes.view(torch.uint8)
    x = buf.view(torch.float8_e4m3fn)[:, 16:16 + n]
    apart = torch.full((2 * T, 13), float("nan"), device=DEV)
    apart[::2, 1:12:2] = scale
    for s in (scale, scale.contiguous(), apart[::2, 1:12:2]):
        assert torch.equal(ex.linear8(x, w, ws, s, transposed=tr), want)
    one = scale[:1].expand(T, -1)
    assert one.stride(0) == 0 or T == 1
    assert torch.equal(ex.linear8(x, w, ws, one, transposed=tr), ex.linear8(codes, w, ws, one.contiguous(), transposed=tr))
    with pytest.raises(ex.Exl3Error, match="aligned|multiple"):
        ex.linear8(buf.view(torch.float8_e4m3fn)[:, 8:8 + n], w, ws, scale, transposed=tr)


def test_expert_layers_of_threads_that_call_at_once(ex):
    """Six host threads, each with its stream, type, bits and tile size."""
    import threading
    from test_gpu_expert_layer import Experts, a_router
    from test_gpu_linear import DT
    jobs = []
    for i in range(6):
        g, dt = gen(30 + i), ("bf16", "fp16")[i % 2]
        m = Experts(g, 12, 256 + 128 * i, 384, 1 + i % 4, 1 + (i + 1) % 4, i % 3 == 0)
        x = acts(g, (1, 8, 30, 64, 100, 256)[i], m.H, dt)
        jobs.append((m, x, a_router(g, 12, m.H, DT[dt])))
    want = [m.run(ex, x, 4, router=r) for m, x, r in jobs]
    torch.cuda.synchronize()
    other = []

    def run(i):
        m, x, r = jobs[i]
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = m.run(ex, x, 4, router=r)
                s.synchronize()
                if not torch.equal(got, want[i]):
                    other.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not other
    # six threads that launch into one stream, each with its workspace
    def one_stream(i):
        m, x, r = jobs[i]
        for _ in range(20):
            got.append((i, m.run(ex, x, 4, router=r)))

    got = []
    threads = [threading.Thread(target=one_stream, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(got) == 120 and all(torch.equal(y, want[i]) for i, y in got)
