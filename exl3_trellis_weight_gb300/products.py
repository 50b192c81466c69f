"""Products with trellis-coded matrices: one shared projection with the low-rank
adapters of many requests (``linear``, ``linear_backward``) and products grouped
by expert (``expert_linear``).  The same thin binding as the package's other
entry points; a call that decodes a single token is a few microseconds of GPU
work, so the checks here stay few and cheap."""
from __future__ import annotations

import torch

from . import EXL3_BF16, EXL3_F16, Exl3Error, lib

_DT = {torch.bfloat16: EXL3_BF16, torch.float16: EXL3_F16}
_fn = None


# the current stream's handle, without a Stream object around it (a microsecond)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _lib():
    global _fn
    if _fn is None:
        _fn = lib()
    return _fn


def _fail(status: int):
    L = _lib()
    raise Exl3Error(status, f"{L.exl3_status_str(status).decode()}: {L.exl3_last_error().decode()}")


def _call(entry, index, *args):
    """The entry point with CUDA device ``index`` current: the library launches on the
    current device, which need not be the tensors'."""
    if _current_device() == index:
        st = entry(*args)
    else:
        with torch.cuda.device(index):
            st = entry(*args)
    if st:
        _fail(st)


def linear_workspace_bytes(T: int, rows: int, cols: int, transposed: bool = False, n_adapters: int = 0,
                           rank: int = 0) -> int:
    return int(_lib().exl3_linear_workspace_bytes(T, rows, cols, int(transposed), n_adapters, rank))


def linear_backward_workspace_bytes(T: int, rows: int, cols: int, transposed: bool = False, n_adapters: int = 0,
                                    rank: int = 0) -> int:
    return int(_lib().exl3_linear_backward_workspace_bytes(T, rows, cols, int(transposed), n_adapters, rank))


def expert_linear_workspace_bytes(T: int, rows: int, cols: int, transposed: bool = False) -> int:
    return int(_lib().exl3_expert_linear_workspace_bytes(T, rows, cols, int(transposed)))


def _activations(t, name, columns, like=None):
    """Row stride of a [T, columns] tensor, in elements."""
    shape = t.shape
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    if len(shape) != 2 or shape[1] != columns:
        raise ValueError(f"{name} must be [tokens, {columns}], got {tuple(shape)}")
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype} of {name} (bfloat16 or float16)")
    if like is not None and (t.dtype != like.dtype or shape[0] != like.shape[0] or t.device != like.device):
        raise ValueError(f"{name} must have the dtype, tokens and device of the activations")
    row, column = t.stride()
    if column != 1 and shape[0]:
        raise ValueError(f"{name}'s columns must be contiguous")
    return row if shape[0] > 1 else columns


def _dense(t, name, dtype, shape, index):
    """Address of a contiguous tensor of this type and shape on CUDA device `index`."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on CUDA device {index} (no CPU fallback)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _coded(codes, su, sv, K, scale, lead, device):
    """Pointers of a coded matrix (or a stack of them) and its two sizes."""
    shape, index = codes.shape, device.index if device.type == "cuda" else -1
    if len(shape) != len(lead) + 3:
        raise ValueError(f"codes must have {len(lead) + 3} dimensions, got {tuple(shape)}")
    if codes.dtype is not torch.int16:
        raise ValueError(f"codes must be int16, got {codes.dtype}")
    rows, cols = shape[-3] * 16, shape[-2] * 16
    c = _dense(codes, "codes", torch.int16, (*lead, shape[-3], shape[-2], 16 * K), index)
    if not isinstance(scale, torch.Tensor):
        scale = torch.full(lead, float(scale), dtype=torch.float32, device=device)
    u = _dense(su, "su", torch.float32, (*lead, rows), index)
    v = _dense(sv, "sv", torch.float32, (*lead, cols), index)
    # the scale's tensor is returned too: one made here must live until the launch
    return rows, cols, c, u, v, _dense(scale, "scale", torch.float32, lead, index), scale


_NO_ADAPTERS = (None, None, None, None, None, 0, 0)


def _adapters(A, B, gain, slots, ranks, n_in, n_out, x):
    if A is None:
        if B is not None or gain is not None or slots is not None or ranks is not None:
            raise ValueError("B, gain, slots and ranks need A")
        return _NO_ADAPTERS
    if B is None or gain is None or slots is None:
        raise ValueError("A needs B, gain and slots")
    if A.dim() != 3:
        raise ValueError(f"A must be [adapters, rank, {n_in}], got {tuple(A.shape)}")
    dev, dt = x.get_device(), x.dtype
    n, r, _ = A.shape
    return (_dense(A, "A", dt, (n, r, n_in), dev), _dense(B, "B", dt, (n, r, n_out), dev),
            _dense(gain, "gain", torch.float32, (n,), dev),
            _dense(slots, "slots", torch.int32, (x.shape[0],), dev),
            None if ranks is None else _dense(ranks, "ranks", torch.int32, (n,), dev), n, r)


def _ws(need, device, ws):
    if ws is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous CUDA tensor")
    if ws.get_device() != device.index:
        raise ValueError(f"the workspace must be on CUDA device {device.index}, as the other tensors")
    return ws


_grad_on = torch.is_grad_enabled


def _refuse_lost(out, **constants):
    """For a call that goes through autograd: raises where a gradient would be lost."""
    for name, t in constants.items():
        if t is not None and t.requires_grad:
            raise ValueError(f"there is no gradient with respect to {name} (detach it)")
    if out is not None:
        raise ValueError("out does not go with inputs that want a gradient (torch.no_grad() lets it)")


# Results go to addresses, which autograd does not see: a tensor given for one may not be part of a
# graph of gradients (as with torch's own out=), and behind the call its version says that it was
# overwritten, so that a backward pass that had saved it raises.
_overwritten = torch.autograd.graph.increment_version


def _refuse_graph(t, name):
    if t.requires_grad and _grad_on():
        raise ValueError(f"{name} wants a gradient, which would be lost (detach it, or torch.no_grad() lets it)")


# whether forward-mode derivatives are on their way at all (a private name of torch's, read so
# that a call outside of them pays nothing; without it every tensor is asked)
def _forward():
    return getattr(torch.autograd.forward_ad, "_current_level", 0) >= 0


def _refuse_tangents(**inputs):
    """Raises where a forward-mode derivative would be lost: the library reads addresses."""
    for name, t in inputs.items():
        if isinstance(t, torch.Tensor) and torch.autograd.forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"there is no forward-mode derivative through {name} (only gradients)")


def _rows(t):
    """t with rows as the library takes them (an expanded gradient has none)."""
    return t if t.shape[0] == 0 or (t.stride(1) == 1 and t.stride(0) >= t.shape[1]) else t.contiguous()


class _Linear(torch.autograd.Function):
    """``linear`` with ``linear_backward`` as its gradient."""

    @staticmethod
    def forward(ctx, x, A, B, codes, su, sv, K, scale, transposed, gain, slots, ranks, ws):
        ctx.save_for_backward(None if A is None else x, A, B, codes, su, sv, scale, gain, slots, ranks)
        ctx.coded = K, transposed
        return linear(x, codes, su, sv, K, scale, transposed, A, B, gain, slots, ranks, ws=ws)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, A, B, codes, su, sv, scale, gain, slots, ranks = ctx.saved_tensors
        K, transposed = ctx.coded
        g = linear_backward(_rows(dy), x, codes, su, sv, K, scale, transposed, A, B, gain, slots, ranks)
        return g["dx"], g["dA"], g["dB"], *(None,) * 10


class _ExpertLinear(torch.autograd.Function):
    """``expert_linear`` with the call of the other transposition as its gradient."""

    @staticmethod
    def forward(ctx, x, offsets, codes, su, sv, K, scale, transposed, ws):
        ctx.save_for_backward(offsets, codes, su, sv, scale)
        ctx.coded = K, transposed
        return expert_linear(x, offsets, codes, su, sv, K, scale, transposed, ws=ws)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        offsets, codes, su, sv, scale = ctx.saved_tensors
        K, transposed = ctx.coded
        return expert_linear(_rows(dy), offsets, codes, su, sv, K, scale, not transposed), *(None,) * 8


def linear(x, codes, su, sv, K: int, scale, transposed: bool = False, A=None, B=None, gain=None, slots=None,
           ranks=None, out=None, ws=None):
    """exl3_linear: y = x W^ (transposed: x W^^T) for the matrix coded in ``codes``
    [rows/16, cols/16, 16K], plus each token's low-rank adapter.

    x [T, inputs] bfloat16 or float16 (rows may be strided); su [rows], sv [cols]
    float32; scale a float32 device scalar (as ``quantize`` returns it) or a number.
    A [n, r, inputs], B [n, r, outputs] of x's dtype, gain [n] float32, slots [T]
    int32 (the adapter of each token; out of [0, n): none), ranks [n] int32 or None.
    Returns y [T, outputs] of x's dtype, through which x, A and B get their gradients
    where they want them."""
    dev = x.device
    rows, cols, pc, pu, pv, ps, scale_ = _coded(codes, su, sv, K, scale, (), dev)
    n_in, n_out = (cols, rows) if transposed else (rows, cols)
    xs = _activations(x, "x", n_in)
    T = x.shape[0]
    pA, pB, pg, pslots, pranks, n, r = _adapters(A, B, gain, slots, ranks, n_in, n_out, x)
    if _forward():
        _refuse_tangents(x=x, su=su, sv=sv, scale=scale_, A=A, B=B, gain=gain)
    if _grad_on() and (x.requires_grad or su.requires_grad or sv.requires_grad or scale_.requires_grad or
                       (n and (A.requires_grad or B.requires_grad or gain.requires_grad))):
        _refuse_lost(out, su=su, sv=sv, scale=scale_, gain=gain)
        return _Linear.apply(x, A, B, codes, su, sv, K, scale_, transposed, gain, slots, ranks, ws)
    given = out is not None
    if given:
        ys = _activations(out, "out", n_out, like=x)
        _refuse_graph(out, "out")
    else:
        out = torch.empty(T, n_out, dtype=x.dtype, device=dev)
        ys = n_out
    L = _lib()
    tr = 1 if transposed else 0
    ws = _ws(L.exl3_linear_workspace_bytes(T, rows, cols, tr, n, r), dev, ws)
    _call(L.exl3_linear, dev.index, x.data_ptr(), _DT[x.dtype], T, xs, pc, rows, cols, K, pu, pv, ps, tr, pA, pB, pg,
          pslots, pranks, n, r, out.data_ptr(), ys, ws.data_ptr(), ws.numel() * ws.element_size(), _stream(dev.index))
    if given:
        _overwritten(out)
    return out


def linear_backward(dy, x, codes, su, sv, K: int, scale, transposed: bool = False, A=None, B=None, gain=None,
                    slots=None, ranks=None, dx=None, ws=None):
    """exl3_linear_backward: gradients of ``linear`` for dy [T, outputs], with the
    arguments of the forward call.  Returns dict(dx, dA, dB) (dA, dB None without
    adapters; x is then not needed and may be None)."""
    dev = dy.device
    rows, cols, pc, pu, pv, ps, _keep = _coded(codes, su, sv, K, scale, (), dev)
    n_in, n_out = (cols, rows) if transposed else (rows, cols)
    dys = _activations(dy, "dy", n_out)
    T = dy.shape[0]
    pA, pB, pg, pslots, pranks, n, r = _adapters(A, B, gain, slots, ranks, n_in, n_out, dy)
    if _forward():
        _refuse_tangents(dy=dy, x=x, su=su, sv=sv, scale=_keep, A=A, B=B, gain=gain)
    px, xs = None, n_in
    if n:
        if x is None:
            raise ValueError("the adapters' gradients need x")
        xs = _activations(x, "x", n_in, like=dy)
        px = x.data_ptr()
    dA = torch.empty_like(A) if n else None
    dB = torch.empty_like(B) if n else None
    given = dx is not None
    if given:
        dxs = _activations(dx, "dx", n_in, like=dy)
        _refuse_graph(dx, "dx")
    else:
        dx = torch.empty(T, n_in, dtype=dy.dtype, device=dev)
        dxs = n_in
    L = _lib()
    tr = 1 if transposed else 0
    ws = _ws(L.exl3_linear_backward_workspace_bytes(T, rows, cols, tr, n, r), dev, ws)
    _call(L.exl3_linear_backward, dev.index, dy.data_ptr(), dys, px, xs, _DT[dy.dtype], T, pc, rows, cols, K, pu, pv,
          ps, tr, pA, pB, pg, pslots, pranks, n, r, dx.data_ptr(), dxs, dA.data_ptr() if n else None,
          dB.data_ptr() if n else None, ws.data_ptr(), ws.numel() * ws.element_size(), _stream(dev.index))
    if given:
        _overwritten(dx)
    return dict(dx=dx, dA=dA, dB=dB)


def expert_linear(x, offsets, codes, su, sv, K: int, scale, transposed: bool = False, out=None, ws=None):
    """exl3_expert_linear: rows offsets[e]..offsets[e+1]-1 of x [T, inputs] times the
    matrix of expert e, coded in codes [E, rows/16, cols/16, 16K] with su [E, rows],
    sv [E, cols] and scale [E] (float32 tensors).  offsets: int32 [E + 1] on the
    device, ascending; rows of no expert give 0.  The input gradient is the same
    call with ``transposed`` flipped, and what x gets through autograd.  Returns y
    [T, outputs] of x's dtype."""
    dev = x.device
    if codes.dim() != 4:
        raise ValueError(f"codes must be [experts, rows/16, cols/16, 16K], got {tuple(codes.shape)}")
    E = codes.shape[0]
    rows, cols, pc, pu, pv, ps, scale_ = _coded(codes, su, sv, K, scale, (E,), dev)
    n_in, n_out = (cols, rows) if transposed else (rows, cols)
    xs = _activations(x, "x", n_in)
    T = x.shape[0]
    po = _dense(offsets, "offsets", torch.int32, (E + 1,), x.get_device())
    if _forward():
        _refuse_tangents(x=x, su=su, sv=sv, scale=scale_)
    if _grad_on() and (x.requires_grad or su.requires_grad or sv.requires_grad or scale_.requires_grad):
        _refuse_lost(out, su=su, sv=sv, scale=scale_)
        return _ExpertLinear.apply(x, offsets, codes, su, sv, K, scale_, transposed, ws)
    given = out is not None
    if given:
        ys = _activations(out, "out", n_out, like=x)
        _refuse_graph(out, "out")
    else:
        out = torch.empty(T, n_out, dtype=x.dtype, device=dev)
        ys = n_out
    L = _lib()
    tr = 1 if transposed else 0
    ws = _ws(L.exl3_expert_linear_workspace_bytes(T, rows, cols, tr), dev, ws)
    _call(L.exl3_expert_linear, dev.index, x.data_ptr(), _DT[x.dtype], T, xs, po, E, pc, rows, cols, K, pu, pv, ps, tr,
          out.data_ptr(), ys, ws.data_ptr(), ws.numel() * ws.element_size(), _stream(dev.index))
    if given:
        _overwritten(out)
    return out
