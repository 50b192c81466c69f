"""The device that the encoder's entry points launch on (not gpu): that of their tensors,
whichever one is current.  As in test_linear_device_host.py, tensors only say that they are
on a device and the library notes the current one."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from test_linear_device_host import Elsewhere, Library, Placed, placed  # noqa: E402


@pytest.fixture
def ex(monkeypatch):
    import exl3_trellis_weight_gb300 as ex
    devices = [0]

    @contextlib.contextmanager
    def device(d):
        devices.append(d.index)
        yield
        devices.pop()

    library = Library(devices)
    monkeypatch.setattr(ex, "lib", lambda: library)
    monkeypatch.setattr(ex, "_stream", lambda d: 1000 + d.index)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: devices[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    # results made by the calls come from the host and say the same
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None: empty(*s, dtype=dtype).as_subclass(
        Placed if device.index else Elsewhere))
    ex.seen = library.seen
    return ex


CALLS = {
    "rotate": lambda ex, t: ex.rotate(t(128, 128), t(128), t(128)),
    "encode_tiles": lambda ex, t: ex.encode_tiles(t(128, 128), 2),
    "decode_tiles": lambda ex, t: ex.decode_tiles(t(8, 8, 32, dtype=torch.int16), 128, 128, 2),
    "encode_rows": lambda ex, t: ex.encode_rows(t(4, 256), 2),
    "decode_rows": lambda ex, t: ex.decode_rows(t(4, 32, dtype=torch.int16), 4, 256, 2),
    "mse": lambda ex, t: ex.mse(t(128, 128), t(128, 128)),
    "quantize": lambda ex, t: ex.quantize(t(128, 128), t(128), t(128), 2),
    "gss_scale": lambda ex, t: ex.gss_scale(t(128, 128), t(128), t(128), 2),
    "scale_search": lambda ex, t: ex.scale_search(t(128, 128), t(128), t(128), 2),
    "block_ldl": lambda ex, t: ex.block_ldl(t(128, 128, dtype=torch.float64)),
    "ldlq": lambda ex, t: ex.ldlq(t(128, 128), t(128, 128), 2, 1.0),
    "regularize": lambda ex, t: ex.regularize(t(128, 128), t(128), t(128)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_launches_on_the_device_of_the_tensors(ex, name):
    for cls in (Placed, Elsewhere):
        CALLS[name](ex, lambda *s, dtype=torch.float32: placed(*s, dtype=dtype, cls=cls))
        assert ex.seen == [("exl3_" + name, cls.where, 1000 + cls.where)]
        ex.seen.clear()
