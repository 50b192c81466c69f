"""The device that norms, 8-bit blocks and products and expert layers launch on (not gpu): that
of their tensors, whichever one is current, and what a call refuses because it would lose a
gradient.  The stand-ins are those of the coded products' test."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from test_linear_device_host import Elsewhere, Library, Placed, placed  # noqa: E402

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture
def layer(monkeypatch):
    from exl3_trellis_weight_gb300 import layer, products
    devices = [0]

    @contextlib.contextmanager
    def device(index):
        devices.append(index if isinstance(index, int) else index.index)
        yield
        devices.pop()

    def maker(index):
        return lambda shape, stride, dtype: torch.empty_strided(shape, stride, dtype=dtype).as_subclass(Placed if index == 1 else Elsewhere)

    monkeypatch.setattr(products, "_fn", Library(devices))
    monkeypatch.setattr(products, "_current_device", lambda: devices[-1], raising=False)
    for module in (products, layer):
        monkeypatch.setattr(module, "_stream", lambda index: 1000 + index)
    monkeypatch.setattr(layer, "_maker", maker)
    monkeypatch.setattr(torch.cuda, "device", device)
    layer.seen, layer.devices = products._fn.seen, devices
    return layer


def tensors(cls):
    def t(*s, dtype=torch.float32):
        return placed(*s, dtype=dtype, cls=cls)
    up = t(3, 16, 8, 32, dtype=torch.int16), t(3, 256), t(3, 128), t(3)
    down = t(3, 8, 16, 32, dtype=torch.int16), t(3, 128), t(3, 256), t(3)
    return dict(x=t(2, 256, dtype=BF16), r=t(2, 256, dtype=BF16), w=t(256), w8=t(256, 128, dtype=E4M3), s8=t(2, 1), x8=t(2, 256, dtype=E4M3),
                xs=t(2, 2), up=up, down=down, router=t(3, 256), ids=t(2, 1, dtype=torch.int32), pw=t(2, 1), ws=t(256, dtype=torch.uint8))


def calls(m, v):
    return {"rms_norm": lambda: m.rms_norm(v["x"], v["w"], residual=v["r"], want_y8=True),
            "rms_norm_backward": lambda: m.rms_norm_backward(v["x"], v["r"], v["w"], ws=v["ws"]),
            "quantize8": lambda: m.quantize8(v["x"]),
            "linear8": lambda: m.linear8(v["x"], v["w8"], v["s8"], ws=v["ws"]),
            "expert_layer": lambda: m.expert_layer(v["x"], v["up"], v["up"], v["down"], 2, 1, router=v["router"], ws=v["ws"])}


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_backward", "quantize8", "linear8", "expert_layer"])
def test_launches_on_the_device_of_the_tensors(layer, name):
    for cls in (Placed, Elsewhere):
        calls(layer, tensors(cls))[name]()
        assert layer.seen == [("exl3_" + name, cls.where, 1000 + cls.where)]
        assert layer.devices == [0]
        layer.seen.clear()


@pytest.mark.parametrize("name,key", [("rms_norm", "w"), ("rms_norm", "r"), ("rms_norm_backward", "r"), ("rms_norm_backward", "w"),
                                      ("rms_norm_backward", "ws"), ("linear8", "w8"), ("linear8", "s8"), ("linear8", "ws"), ("expert_layer", "up"),
                                      ("expert_layer", "down"), ("expert_layer", "router"), ("expert_layer", "ws"), ("expert_layer", "x")])
def test_refuses_tensors_of_several_devices(layer, name, key):
    v = tensors(Placed)
    v[key] = tensors(Elsewhere)[key]
    with pytest.raises(ValueError):
        calls(layer, v)[name]()
    assert not layer.seen


def test_refuses_what_would_lose_a_gradient(layer):
    v = tensors(Placed)

    def wants(t):
        return t.detach().clone().as_subclass(Placed).requires_grad_()

    def norm(**kw):
        return layer.rms_norm(**{**dict(x=v["x"], weight=v["w"], residual=v["r"]), **kw})

    def product(**kw):
        return layer.linear8(**{**dict(x=v["x"], w=v["w8"], w_scale=v["s8"], ws=v["ws"]), **kw})

    def experts(**kw):
        return layer.expert_layer(**{**dict(x=v["x"], gate=v["up"], up=v["up"], down=v["down"], K=2, top_k=1, router=v["router"], ws=v["ws"]), **kw})

    def with_part(i):
        return tuple(wants(t) if j == i else t for j, t in enumerate(v["up"]))

    y = placed(2, 256, dtype=BF16)
    given = dict(router=None, ids=v["ids"])
    for call, bad in ((norm, dict(x=wants(v["x"]), want_y8=True)), (norm, dict(weight=wants(v["w"]), out=y)), (norm, dict(residual=wants(v["r"]), h=y)),
                      (product, dict(w_scale=wants(v["s8"]))), (product, dict(x=wants(v["x"]), out=placed(2, 128, dtype=BF16))),
                      (product, dict(x=v["x8"], x_scale=wants(v["xs"]))),
                      (experts, dict(x=wants(v["x"]))), (experts, dict(router=wants(v["router"]))), (experts, dict(given, weights=wants(v["pw"]))),
                      (experts, dict(gate=with_part(1))), (experts, dict(up=with_part(2))), (experts, dict(gate=with_part(3)))):
        with pytest.raises(ValueError, match="gradient"):
            call(**bad)
        assert not layer.seen
        with torch.no_grad():
            call(**bad)
        assert len(layer.seen) == 1
        layer.seen.clear()


def test_an_expert_scale_may_be_a_number(layer):
    v = tensors(Placed)
    new = torch.full

    def full(shape, value, dtype, device):
        return new(shape, value, dtype=dtype).as_subclass(Placed)

    layer.torch.full, keep = full, layer.torch.full
    try:
        layer.expert_layer(v["x"], (*v["up"][:3], 0.5), v["up"], v["down"], 2, 1, router=v["router"], ws=v["ws"])
    finally:
        layer.torch.full = keep
    assert len(layer.seen) == 1


def test_refuses_gradients_of_8_bit_blocks_and_matrices(layer):
    """A torch.nn.Parameter in e4m3 wants a gradient unless told otherwise, and none comes to it."""
    v = tensors(Placed)

    def wants(t):
        return t.detach().clone().as_subclass(Placed).requires_grad_()

    for call in (lambda: layer.quantize8(wants(v["x"])), lambda: layer.quantize8(wants(v["w"][None]), block_rows=128),
                 lambda: layer.linear8(v["x"], wants(v["w8"]), v["s8"], ws=v["ws"]),
                 lambda: layer.linear8(wants(v["x"]), wants(v["w8"]), v["s8"], ws=v["ws"]),
                 lambda: layer.linear8(v["x8"], wants(v["w8"]), v["s8"], v["xs"])):
        with pytest.raises(ValueError, match="gradient"):
            call()
        assert not layer.seen
        with torch.no_grad():
            call()
        assert len(layer.seen) == 1
        layer.seen.clear()
    # what wants none goes through, in either mode
    layer.quantize8(v["x"])
    layer.linear8(v["x"], torch.nn.Parameter(v["w8"].as_subclass(torch.Tensor), requires_grad=False).as_subclass(Placed), v["s8"], ws=v["ws"])
    assert len(layer.seen) == 2


def test_refuses_what_would_lose_a_tangent(layer):
    """Forward-mode derivatives: a tensor that carries one does not want a gradient, so it has to be
    asked.  The same calls go through outside of forward mode, and inside it without tangents."""
    from torch.autograd import forward_ad as fw
    from exl3_trellis_weight_gb300 import products
    v = tensors(Placed)
    one = dict(zip(("codes", "su", "sv", "scale"), (t[0] for t in v["up"])))
    A, B, gain = placed(1, 4, 256, dtype=BF16), placed(1, 4, 128, dtype=BF16), placed(1)
    slots, y, offsets = placed(2, dtype=torch.int32), placed(2, 128, dtype=BF16), placed(4, dtype=torch.int32)

    def grouped(**kw):
        m = dict(zip(("codes", "su", "sv", "scale"), v["up"]))
        return products.expert_linear(**{**dict(x=v["x"], offsets=offsets, K=2, out=y, ws=v["ws"]), **m, **kw})

    def linear(**kw):
        return products.linear(**{**dict(x=v["x"], K=2, A=A, B=B, gain=gain, slots=slots, out=y, ws=v["ws"]), **one, **kw})

    def backward(**kw):
        a = dict(dy=y, x=v["x"], K=2, A=A, B=B, gain=gain, slots=slots, dx=placed(2, 256, dtype=BF16), ws=v["ws"])
        return products.linear_backward(**{**a, **one, **kw})

    def norm(**kw):
        return layer.rms_norm(**{**dict(x=v["x"], weight=v["w"], residual=v["r"]), **kw})

    def norm_backward(**kw):
        return layer.rms_norm_backward(**{**dict(dy=v["x"], h=v["r"], weight=v["w"], dh=v["r"], ws=v["ws"]), **kw})

    def product(**kw):
        return layer.linear8(**{**dict(x=v["x"], w=v["w8"], w_scale=v["s8"], ws=v["ws"]), **kw})

    def experts(**kw):
        return layer.expert_layer(**{**dict(x=v["x"], gate=v["up"], up=v["up"], down=v["down"], K=2, top_k=1, router=v["router"], ws=v["ws"]), **kw})

    def part(i):
        return lambda d: tuple(d if j == i else t for j, t in enumerate(v["up"]))

    given = dict(router=None, ids=v["ids"])
    cases = [(norm, "x", v["x"]), (norm, "weight", v["w"]), (norm, "residual", v["r"]), (norm_backward, "dy", v["x"]), (norm_backward, "h", v["r"]),
             (norm_backward, "weight", v["w"]), (norm_backward, "dh", v["r"]), (layer.quantize8, "x", v["x"]), (product, "x", v["x"]),
             (product, "w_scale", v["s8"]), (experts, "x", v["x"]), (experts, "router", v["router"]), (linear, "x", v["x"]), (linear, "A", A),
             (linear, "B", B), (linear, "gain", gain), (linear, "su", one["su"]), (linear, "scale", one["scale"]), (backward, "dy", y),
             (backward, "x", v["x"]), (backward, "A", A), (grouped, "x", v["x"]), (grouped, "sv", v["up"][2])]
    calls = [(lambda d, call=call, key=key: call(**{key: d}), t) for call, key, t in cases]
    calls += [(lambda d: product(x=v["x8"], x_scale=d), v["xs"]), (lambda d: experts(**given, weights=d), v["pw"])]
    calls += [(lambda d, i=i: experts(up=part(i)(d)), v["up"][i]) for i in (1, 2, 3)]
    for call, t in calls:
        with fw.dual_level():
            for grad in (torch.enable_grad, torch.no_grad):
                with grad(), pytest.raises(ValueError, match="forward-mode"):
                    call(fw.make_dual(t, torch.ones_like(t)))
            assert not layer.seen
            call(t)
        call(t)
        assert len(layer.seen) == 2
        layer.seen.clear()


def outputs(layer):
    """Each call with a tensor given for a result: (call, a tensor that it may be)."""
    from exl3_trellis_weight_gb300 import products
    v = tensors(Placed)
    one, grouped = dict(zip(("codes", "su", "sv", "scale"), (t[0] for t in v["up"]))), dict(zip(("codes", "su", "sv", "scale"), v["up"]))
    narrow, wide, ws = placed(2, 128, dtype=BF16), placed(2, 256, dtype=BF16), v["ws"]
    offsets = placed(4, dtype=torch.int32)
    return {"norm h": (lambda t: layer.rms_norm(v["x"], v["w"], residual=v["r"], h=t), wide),
            "norm out": (lambda t: layer.rms_norm(v["x"], v["w"], residual=v["r"], out=t), wide),
            "norm gradient dx": (lambda t: layer.rms_norm_backward(v["x"], v["r"], v["w"], dx=t, ws=ws), wide),
            "8-bit product": (lambda t: layer.linear8(v["x"], v["w8"], v["s8"], out=t, ws=ws), narrow),
            "experts": (lambda t: layer.expert_layer(v["x"], v["up"], v["up"], v["down"], 2, 1, router=v["router"], out=t, ws=ws), wide),
            "linear": (lambda t: products.linear(v["x"], K=2, out=t, ws=ws, **one), narrow),
            "linear gradient dx": (lambda t: products.linear_backward(narrow, None, K=2, dx=t, ws=ws, **one), wide),
            "grouped": (lambda t: products.expert_linear(v["x"], offsets, K=2, out=t, ws=ws, **grouped), narrow)}


@pytest.mark.parametrize("name", ["norm h", "norm out", "norm gradient dx", "8-bit product", "experts", "linear", "linear gradient dx", "grouped"])
def test_autograd_hears_of_what_is_overwritten(layer, name):
    call, like = outputs(layer)[name]
    t = like.clone().as_subclass(Placed)
    before = t._version
    call(t)
    assert t._version > before and len(layer.seen) == 1
    # a backward pass that had saved it, or what it is a part of, raises
    whole = torch.ones(like.shape[0], like.shape[1] + 8, dtype=BF16)
    leaf = torch.ones_like(whole).requires_grad_()
    loss = (leaf * whole).sum()
    call(whole[:, :like.shape[1]].as_subclass(Placed))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    # as an inference tensor it has no version, and needs none
    with torch.inference_mode():
        call(like.clone().as_subclass(Placed))
    # part of a graph itself: refused, unless nobody wants gradients
    layer.seen.clear()
    bad = like.clone().as_subclass(Placed).requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(bad)
    assert not layer.seen
    with torch.no_grad():
        call(bad)
    assert len(layer.seen) == 1


def test_a_refused_call_leaves_versions_alone(layer):
    v = tensors(Placed)
    t = placed(2, 256, dtype=BF16)
    before = t._version
    with pytest.raises(ValueError):
        layer.rms_norm(v["x"], v["w"], residual=v["r"], h=t, out=placed(3, 256, dtype=BF16))
    assert t._version == before
