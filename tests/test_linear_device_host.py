"""The device that the products with coded matrices launch on (not gpu): that of their
tensors, whichever one is current.  Tensors here only say that they are on a device, the
library is a stand-in that notes the current one."""
import contextlib

import pytest

torch = pytest.importorskip("torch")


class Placed(torch.Tensor):
    """A host tensor that says it is on CUDA device `where`."""
    where = 1
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.where))

    def get_device(self):
        return self.where


class Elsewhere(Placed):
    where = 0


class Library:
    def __init__(self, devices):
        self.devices, self.seen = devices, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 256
        return lambda *a: self.seen.append((name, self.devices[-1], a[-1])) or 0


@pytest.fixture
def products(monkeypatch):
    from exl3_trellis_weight_gb300 import products
    devices = [0]

    @contextlib.contextmanager
    def device(index):
        devices.append(torch.device("cuda", index).index if isinstance(index, int) else index.index)
        yield
        devices.pop()

    monkeypatch.setattr(products, "_fn", Library(devices))
    monkeypatch.setattr(products, "_stream", lambda index: 1000 + index)
    monkeypatch.setattr(products, "_current_device", lambda: devices[-1], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    products.devices = devices
    return products


def placed(*shape, dtype=torch.float32, cls=Placed):
    return torch.zeros(shape, dtype=dtype).as_subclass(cls)


def calls(products, cls):
    """The three calls with every tensor on the device of `cls`."""
    def t(*s, dtype=torch.float32):
        return placed(*s, dtype=dtype, cls=cls)
    bf16 = torch.bfloat16
    x, y = t(2, 256, dtype=bf16), t(2, 128, dtype=bf16)
    w = t(16, 8, 32, dtype=torch.int16), t(256), t(128), 2, t()
    e = t(1, 16, 8, 32, dtype=torch.int16), t(1, 256), t(1, 128), 2, t(1)
    return {"linear": lambda ws: products.linear(x, *w, out=y, ws=ws),
            "linear_backward": lambda ws: products.linear_backward(y, None, *w, dx=x, ws=ws),
            "expert_linear": lambda ws: products.expert_linear(x, t(2, dtype=torch.int32), *e, out=y, ws=ws)}


@pytest.mark.parametrize("name", ["linear", "linear_backward", "expert_linear"])
def test_launches_on_the_device_of_the_tensors(products, name):
    for cls in (Placed, Elsewhere):
        calls(products, cls)[name](placed(256, dtype=torch.uint8, cls=cls))
        assert products._fn.seen == [("exl3_" + name, cls.where, 1000 + cls.where)]
        assert products.devices == [0]
        products._fn.seen.clear()


@pytest.mark.parametrize("name", ["linear", "linear_backward", "expert_linear"])
def test_refuses_a_workspace_of_another_device(products, name):
    with pytest.raises(ValueError, match="workspace"):
        calls(products, Placed)[name](placed(256, dtype=torch.uint8, cls=Elsewhere))
    assert not products._fn.seen


def test_refuses_what_would_lose_a_gradient(products):
    """A result written to `out`, and factors whose gradients nobody computes."""
    bf16 = torch.bfloat16
    x, y, ws = placed(2, 256, dtype=bf16), placed(2, 128, dtype=bf16), placed(256, dtype=torch.uint8)
    codes, su, sv, s = placed(16, 8, 32, dtype=torch.int16), placed(256), placed(128), placed()
    ad = dict(A=placed(1, 4, 256, dtype=bf16), B=placed(1, 4, 128, dtype=bf16), gain=placed(1), slots=placed(2, dtype=torch.int32))
    e = dict(offsets=placed(2, dtype=torch.int32), codes=codes[None], su=su[None], sv=sv[None], scale=s[None])

    def wants(t):
        return t.detach().clone().as_subclass(Placed).requires_grad_()

    def linear(**kw):
        return products.linear(**{**dict(x=x, codes=codes, su=su, sv=sv, K=2, scale=s, out=y, ws=ws), **ad, **kw})

    def experts(**kw):
        return products.expert_linear(**{**dict(x=x, K=2, out=y, ws=ws), **e, **kw})

    linear(), experts()
    assert len(products._fn.seen) == 2
    for call, bad in ((linear, dict(x=wants(x))), (linear, dict(A=wants(ad["A"]))), (linear, dict(B=wants(ad["B"]))),
                      (linear, dict(gain=wants(ad["gain"]))), (linear, dict(su=wants(su))), (linear, dict(sv=wants(sv))),
                      (linear, dict(scale=wants(s))), (experts, dict(x=wants(x))), (experts, dict(su=wants(e["su"]))),
                      (experts, dict(sv=wants(e["sv"]))), (experts, dict(scale=wants(e["scale"])))):
        with pytest.raises(ValueError, match="gradient"):
            call(**bad)
        with torch.no_grad():
            call(**bad)
    assert len(products._fn.seen) == 2 + 11
