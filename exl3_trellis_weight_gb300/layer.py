"""What stands around the products of a layer: root-mean-square norms with the
residual's addition (``rms_norm``, ``rms_norm_backward``), blocks in 8 bits
(``quantize8``) and products with them (``linear8``), and whole mixture-of-experts
layers for a few tokens (``expert_layer``).  The same thin binding as ``products``,
whose helpers it uses."""
from __future__ import annotations

import ctypes

import torch

from . import EXL3_BF16, EXL3_E4M3, EXL3_F16, EXL3_F32
from .products import (_activations, _call, _current_device, _dense, _forward, _grad_on, _lib, _overwritten, _refuse_graph,
                       _refuse_tangents, _rows, _stream)
from .products import _ws as _given_ws

_DT = {torch.bfloat16: EXL3_BF16, torch.float16: EXL3_F16}
_DT_X = {**_DT, torch.float32: EXL3_F32}
_E4M3 = torch.float8_e4m3fn

# torch.empty_strided without the dispatcher, on the current device (two microseconds of
# the seven that an allocation and a launch take)
_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _maker(index):
    """make(shape, stride, dtype) -> an uninitialised tensor on CUDA device `index`."""
    if _strided is not None and _current_device() == index:
        return _strided
    dev = torch.device("cuda", index) if index >= 0 else torch.device("cpu")
    return lambda shape, stride, dtype: torch.empty_strided(shape, stride, dtype=dtype, device=dev)


def _ws(need, dev, ws, make):
    return make((need if need > 256 else 256,), (1,), torch.uint8) if ws is None else _given_ws(need, dev, ws)


def rms_norm_backward_workspace_bytes(T: int, n: int) -> int:
    return int(_lib().exl3_rms_norm_backward_workspace_bytes(T, n))


def linear8_workspace_bytes(T: int, rows: int, cols: int, transposed: bool = False) -> int:
    return int(_lib().exl3_linear8_workspace_bytes(T, rows, cols, int(transposed)))


def expert_layer_workspace_bytes(T: int, hidden: int, inner: int, n_experts: int, top_k: int) -> int:
    return int(_lib().exl3_expert_layer_workspace_bytes(T, hidden, inner, n_experts, top_k))


def _matrix(t, name, dtypes, columns=None, like=None):
    """Row stride of a [T, columns] tensor of one of these types, in elements."""
    shape = t.shape
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    if len(shape) != 2 or (columns is not None and shape[1] != columns):
        raise ValueError(f"{name} must be [tokens, {'columns' if columns is None else columns}], got {tuple(shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"unsupported dtype {t.dtype} of {name}")
    if like is not None and (t.dtype != like.dtype or shape[0] != like.shape[0] or t.device != like.device):
        raise ValueError(f"{name} must have the dtype, tokens and device of the activations")
    row, column = t.stride()
    if column != 1 and shape[0] and shape[1] > 1:
        raise ValueError(f"{name}'s columns must be contiguous")
    return row if shape[0] > 1 else shape[1]


def _like(t, name, shape, x, index):
    """Row stride of a tensor that has x's type, shape and device."""
    if t.dtype is x.dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
        return shape[1]
    return _matrix(t, name, _DT, shape[1], like=x)


def _norm_weight(weight, n, x):
    if weight.dtype is not torch.float32 and weight.dtype is not x.dtype:
        raise ValueError(f"weight must be float32 or {x.dtype}, got {weight.dtype}")
    return _dense(weight, "weight", weight.dtype, (n,), x.get_device()), _DT_X[weight.dtype]


class _RmsNorm(torch.autograd.Function):
    """``rms_norm`` with ``rms_norm_backward`` as its gradient: (y, h), or y without residual."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        r = rms_norm(x, weight, eps, residual)
        ctx.save_for_backward(x if residual is None else r["h"], weight)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return r["y"] if residual is None else (r["y"], r["h"])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        want_x, want_w, want_r, _ = ctx.needs_input_grad
        if dy is None:
            # only h was used
            dx, dw = dh, torch.zeros_like(weight) if want_w and dh is not None else None
        else:
            g = rms_norm_backward(_rows(dy), h, weight, ctx.eps, dh=None if dh is None else _rows(dh), want_dweight=want_w)
            dx, dw = g["dx"], g["dweight"]
        return dx if want_x else None, dw, dx if want_r else None, None


def rms_norm(x, weight, eps: float = 1e-6, residual=None, want_y: bool = True, want_y8: bool = False, h=None, out=None):
    """exl3_rms_norm: h = x + residual (rounded to their dtype), y = h weight /
    sqrt(mean(h^2) + eps) for each row.

    x, residual [T, n] bfloat16 or float16 (rows may be strided), n up to 32768;
    weight [n] of x's dtype or float32; eps a positive normal number.  Returns dict(h, y, y8, scale): h with a
    residual, y with ``want_y``, and with ``want_y8`` y in float8_e4m3fn [T, n]
    with the scale of each 128 columns of a row [T, ceil(n / 128)] (what ``linear8``
    takes); None otherwise.  h may be given as an output (x or residual itself, too),
    ``out`` for y.  x, residual and weight get their gradients through y and h."""
    xs = _matrix(x, "x", _DT)
    shape, index = x.shape, x.get_device()
    T, n = shape
    pw, wdt = _norm_weight(weight, n, x)
    rs = hs = ys = n
    if residual is not None:
        rs = _like(residual, "residual", shape, x, index)
    elif h is not None:
        raise ValueError("h needs a residual (without one it is x)")
    if not (want_y or want_y8):
        raise ValueError("neither y nor y8 is wanted")
    if out is not None and not want_y:
        raise ValueError("out goes with want_y")
    if _forward():
        _refuse_tangents(x=x, weight=weight, residual=residual)
    if _grad_on() and (x.requires_grad or weight.requires_grad or (residual is not None and residual.requires_grad)):
        if want_y8:
            raise ValueError("there is no gradient through y8 (torch.no_grad() lets it)")
        if out is not None or h is not None:
            raise ValueError("out and h do not go with inputs that want a gradient (torch.no_grad() lets them)")
        r = _RmsNorm.apply(x, weight, residual, eps)
        y, h = (r, None) if residual is None else r
        return dict(h=h, y=y, y8=None, scale=None)
    make = _maker(index)
    given = []
    if residual is not None:
        if h is None:
            h = make((T, n), (n, 1), x.dtype)
        else:
            hs = _like(h, "h", shape, x, index)
            _refuse_graph(h, "h")
            given.append(h)
    y = y8 = scale = ph = py = pq = ps = None
    if want_y:
        if out is None:
            y = make((T, n), (n, 1), x.dtype)
        else:
            y = out
            ys = _like(out, "out", shape, x, index)
            _refuse_graph(out, "out")
            given.append(out)
        py = y.data_ptr()
    if want_y8:
        y8 = make((T, n), (n, 1), _E4M3)
        scale = make((T, (n + 127) // 128), (1, T), torch.float32)
        pq, ps = y8.data_ptr(), scale.data_ptr()
    if h is not None:
        ph = h.data_ptr()
    _call(_lib().exl3_rms_norm, index, x.data_ptr(), _DT[x.dtype], T, n, xs, None if residual is None else residual.data_ptr(),
          rs, pw, wdt, eps, ph, hs, py, ys, pq, ps, _stream(index))
    if given:
        _overwritten(given)
    return dict(h=h, y=y, y8=y8, scale=scale)


def rms_norm_backward(dy, h, weight, eps: float = 1e-6, dh=None, want_dweight: bool = True, dx=None, ws=None):
    """exl3_rms_norm_backward: gradients of ``rms_norm``'s y for dy [T, n]; h is the
    forward's h (x without a residual), dh the gradient of h's other uses or None.
    Returns dict(dx, dweight): dx is the gradient of x and of the residual (dy or dh
    itself may be given for it), dweight has weight's dtype (None without
    ``want_dweight``)."""
    gs = _matrix(dy, "dy", _DT)
    shape, index = dy.shape, dy.get_device()
    T, n = shape
    hs = _like(h, "h", shape, dy, index)
    pw, wdt = _norm_weight(weight, n, dy)
    ds = xs = n
    if dh is not None:
        ds = _like(dh, "dh", shape, dy, index)
    if _forward():
        _refuse_tangents(dy=dy, h=h, weight=weight, dh=dh)
    make = _maker(index)
    given = dx is not None
    if given:
        xs = _like(dx, "dx", shape, dy, index)
        _refuse_graph(dx, "dx")
    else:
        dx = make((T, n), (n, 1), dy.dtype)
    L = _lib()
    dw = pd = pws = None
    bytes_ = 0
    if want_dweight:
        dw = make((n,), (1,), weight.dtype)
        ws = _ws(L.exl3_rms_norm_backward_workspace_bytes(T, n), dy.device, ws, make)
        pd, pws, bytes_ = dw.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size()
    _call(L.exl3_rms_norm_backward, index, dy.data_ptr(), gs, h.data_ptr(), hs, _DT[dy.dtype], T, n, pw, wdt, eps,
          None if dh is None else dh.data_ptr(), ds, dx.data_ptr(), xs, pd, pws, bytes_, _stream(index))
    if given:
        _overwritten(dx)
    return dict(dx=dx, dweight=dw)


def quantize8(x, block_rows: int = 1):
    """exl3_quantize8: x [T, n] (bfloat16, float16 or float32, rows may be strided)
    -> (codes float8_e4m3fn [T, n], scale float32): codes times the scale of their
    block of ``block_rows`` x 128 stand for x.  block_rows 1, for activations: scale
    [T, ceil(n / 128)]; 128, for weights: [ceil(T / 128), ceil(n / 128)].  There is no
    gradient through it: an x that wants one is refused (torch.no_grad() lets it)."""
    xs = _matrix(x, "x", _DT_X)
    if _forward():
        _refuse_tangents(x=x)
    if _grad_on() and x.requires_grad:
        raise ValueError("there is no gradient through 8-bit blocks (detach x, or torch.no_grad() lets it)")
    T, n = x.shape
    index = x.get_device()
    make = _maker(index)
    codes = make((T, n), (n, 1), _E4M3)
    nb = (n + 127) // 128
    if block_rows == 1:
        scale = make((T, nb), (1, T), torch.float32)
    else:
        scale = make(((T + 127) // 128, nb), (nb, 1), torch.float32)
    _call(_lib().exl3_quantize8, index, x.data_ptr(), _DT_X[x.dtype], T, n, xs, block_rows, codes.data_ptr(),
          scale.data_ptr(), _stream(index))
    return codes, scale


class _Linear8(torch.autograd.Function):
    """``linear8`` with the call of the other transposition as its gradient."""

    @staticmethod
    def forward(ctx, x, w, w_scale, transposed, dtype, ws):
        ctx.save_for_backward(w, w_scale)
        ctx.transposed, ctx.dtype = transposed, x.dtype
        return linear8(x, w, w_scale, transposed=transposed, dtype=dtype, ws=ws)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        w, w_scale = ctx.saved_tensors
        return linear8(_rows(dy), w, w_scale, transposed=not ctx.transposed, dtype=ctx.dtype), *(None,) * 5


def linear8(x, w, w_scale, x_scale=None, transposed: bool = False, dtype=None, out=None, ws=None):
    """exl3_linear8: y = x W (transposed: x W^T), W in float8_e4m3fn [rows, cols] with
    a float32 scale for each 128 x 128 [ceil(rows / 128), ceil(cols / 128)]; rows and
    cols multiples of 16.

    x [T, inputs] in float8_e4m3fn with ``x_scale`` [T, ceil(inputs / 128)] float32 (any
    strides; rows of x 16-byte aligned), as ``rms_norm`` and ``quantize8`` leave them, or
    in bfloat16 or float16, which are brought to that first.  Returns y [T, outputs] of
    ``dtype`` (bfloat16 or float16; x's own if it is one of them, else bfloat16).  The
    input gradient is the same call with ``transposed`` flipped, and what x in 16 bits
    gets through autograd; w has none, so a w that wants one is refused (a Parameter does
    unless it is made with requires_grad=False)."""
    if w.dim() != 2:
        raise ValueError(f"w must be [rows, cols], got {tuple(w.shape)}")
    rows, cols = w.shape
    n_in, n_out = (cols, rows) if transposed else (rows, cols)
    index = x.get_device()
    pw = _dense(w, "w", _E4M3, (rows, cols), index)
    pws = _dense(w_scale, "w_scale", torch.float32, ((rows + 127) // 128, (cols + 127) // 128), index)
    T = x.shape[0]
    coded = x.dtype is _E4M3
    L = _lib()
    tr = 1 if transposed else 0
    if coded:
        xs, xdt = _matrix(x, "x", (_E4M3,), n_in), EXL3_E4M3
        if x_scale is None:
            raise ValueError("x in float8_e4m3fn needs x_scale")
        if x_scale.dtype is not torch.float32 or x_scale.shape != (T, (n_in + 127) // 128) or x_scale.get_device() != index:
            raise ValueError(f"x_scale must be torch.float32 {(T, (n_in + 127) // 128)} on x's device")
        ps, (st, sb) = x_scale.data_ptr(), x_scale.stride()
    else:
        xs = _matrix(x, "x", _DT, n_in)
        xdt = _DT[x.dtype]
        if x_scale is not None:
            raise ValueError("x_scale goes with x in float8_e4m3fn")
        ps, st, sb = None, 0, 0
    if dtype is None:
        dtype = out.dtype if out is not None else torch.bfloat16 if coded else x.dtype
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype} of y")
    if _forward():
        _refuse_tangents(x=x, w=w, w_scale=w_scale, x_scale=x_scale)
    if _grad_on() and (x.requires_grad or w.requires_grad or w_scale.requires_grad or (x_scale is not None and x_scale.requires_grad)):
        if w.requires_grad or w_scale.requires_grad or coded:
            raise ValueError("there is a gradient only with respect to x in 16 bits (detach w and the scales)")
        if out is not None:
            raise ValueError("out does not go with inputs that want a gradient (torch.no_grad() lets it)")
        return _Linear8.apply(x, w, w_scale, transposed, dtype, ws)
    make = _maker(index)
    given = out is not None
    if given:
        ys = _matrix(out, "out", (dtype,), n_out)
        if out.shape[0] != T or out.get_device() != index:
            raise ValueError("out must have the tokens and device of x")
        _refuse_graph(out, "out")
    else:
        out = make((T, n_out), (n_out, 1), dtype)
        ys = n_out
    pb, nb = None, 0
    if not coded:
        ws = _ws(L.exl3_linear8_workspace_bytes(T, rows, cols, tr), x.device, ws, make)
        pb, nb = ws.data_ptr(), ws.numel() * ws.element_size()
    _call(L.exl3_linear8, index, x.data_ptr(), xdt, T, xs, ps, st, sb, pw, pws, rows, cols, tr, out.data_ptr(), _DT[dtype],
          ys, pb, nb, _stream(index))
    if given:
        _overwritten(out)
    return out


_Experts = ctypes.c_void_p * 12


def expert_layer(x, gate, up, down, K: int, top_k: int, router=None, ids=None, weights=None, transposed: bool = False,
                 K_down: int | None = None, normalize: bool = True, out=None, ws=None):
    """exl3_expert_layer: a mixture-of-experts layer for a few tokens, y_t = sum over the
    token's picks e of w_te (silu(x_t G_e) * (x_t U_e)) D_e.

    x [T, hidden] bfloat16 or float16 (rows may be strided), T up to 256; gate, up, down
    each (codes, su, sv, scale) of all experts as ``expert_linear`` takes them: G and U
    [hidden, inner], D [inner, hidden] (transposed: the other way round, as torch keeps
    them); K bits a weight, ``K_down`` for D where it differs.  Either ``router`` [experts,
    hidden] of x's dtype or float32, from whose softmax the ``top_k`` largest are taken
    (of equals the first; ``normalize``: divided by their sum), or ``ids`` int32 and
    ``weights`` float32 [T, top_k] (an id that is no expert's is passed over).  Returns y
    [T, hidden] of x's dtype.  For more tokens, and for gradients, there is
    ``expert_linear``."""
    index = x.get_device()
    gc = gate[0]
    if gc.dim() != 4:
        raise ValueError(f"gate codes must be [experts, rows/16, cols/16, 16K], got {tuple(gc.shape)}")
    E, rows, cols, _ = gc.shape
    kd = K if K_down is None else K_down
    at, made, grad = [], [], False
    for name, m, r, c, k in (("gate", gate, rows, cols, K), ("up", up, rows, cols, K), ("down", down, cols, rows, kd)):
        if m[0].shape[1:3] != (r, c):
            raise ValueError(f"gate {(16 * rows, 16 * cols)} and {name} {tuple(16 * v for v in m[0].shape[1:3])} do not go together")
        if not isinstance(m[3], torch.Tensor):
            m = (*m[:3], torch.full((E,), float(m[3]), dtype=torch.float32, device=x.device))
            made.append(m)                 # (lives until the launch)
        codes, su, sv, scale = m
        if not (codes.dtype is torch.int16 and codes.shape == (E, r, c, 16 * k) and codes.get_device() == index and codes.is_contiguous()):
            _dense(codes, f"{name} codes", torch.int16, (E, r, c, 16 * k), index)
        if not (su.dtype is torch.float32 and su.shape == (E, 16 * r) and su.get_device() == index and su.is_contiguous()):
            _dense(su, f"{name} su", torch.float32, (E, 16 * r), index)
        if not (sv.dtype is torch.float32 and sv.shape == (E, 16 * c) and sv.get_device() == index and sv.is_contiguous()):
            _dense(sv, f"{name} sv", torch.float32, (E, 16 * c), index)
        if not (scale.dtype is torch.float32 and scale.shape == (E,) and scale.get_device() == index and scale.is_contiguous()):
            _dense(scale, f"{name} scale", torch.float32, (E,), index)
        at += codes.data_ptr(), su.data_ptr(), sv.data_ptr(), scale.data_ptr()
        if su.requires_grad or sv.requires_grad or scale.requires_grad:
            grad = True
    H, F = (cols, rows) if transposed else (rows, cols)
    H, F = 16 * H, 16 * F
    xs = _activations(x, "x", H)
    T = x.shape[0]
    pr = pi = pw = None
    rdt = 0
    if router is not None:
        if ids is not None or weights is not None:
            raise ValueError("ids and weights do not go with a router")
        if router.dtype is not torch.float32 and router.dtype is not x.dtype:
            raise ValueError(f"router must be float32 or {x.dtype}, got {router.dtype}")
        pr, rdt = _dense(router, "router", router.dtype, (E, H), index), _DT_X[router.dtype]
    else:
        if ids is None or weights is None:
            raise ValueError("a router, or ids and weights")
        pi = _dense(ids, "ids", torch.int32, (T, top_k), index)
        pw = _dense(weights, "weights", torch.float32, (T, top_k), index)
    if _forward():
        _refuse_tangents(x=x, router=router, weights=weights)
        for name, m in (("gate", gate), ("up", up), ("down", down)):
            _refuse_tangents(**{f"{name} {part}": t for part, t in zip(("su", "sv", "scale"), m[1:])})
    if _grad_on() and (grad or x.requires_grad or (router is not None and router.requires_grad) or
                       (weights is not None and weights.requires_grad)):
        raise ValueError("there is no gradient through an expert layer (torch.no_grad() lets it; expert_linear has one)")
    make = _maker(index)
    given = out is not None
    if given:
        ys = _activations(out, "out", H, like=x)
        _refuse_graph(out, "out")
    else:
        out = make((T, H), (H, 1), x.dtype)
        ys = H
    L = _lib()
    ws = _ws(L.exl3_expert_layer_workspace_bytes(T, H, F, E, top_k), x.device, ws, make)
    _call(L.exl3_expert_layer, index, x.data_ptr(), _DT[x.dtype], T, xs, pr, rdt, pi, pw, top_k, 1 if normalize else 0, E,
          _Experts(*at), H, F, K, kd, 1 if transposed else 0, out.data_ptr(), ys, ws.data_ptr(),
          ws.numel() * ws.element_size(), _stream(index))
    if given:
        _overwritten(out)
    return out
