"""Cases for the operators that use trellis-coded weights.

Three operators, each with a plain form (elementary torch operations in 32 bits,
rounded once at the end) and the framework's call (``own`` true):

  linear     y = x W^ (or x W^^T) with W^ coded at K bits, plus the low-rank
             adapter of each token's request: y_t += gain_i B_i^T A_i x_t
  backward   of the same with respect to x, A and B (the codes are frozen)
  experts    y[rows of e] = x[rows of e] W^_e for ragged groups of rows

W^ = 2^-7 s diag(su) (H V H) diag(sv): V the codebook levels of the codes, H the
natural-order Sylvester Hadamard matrix on each block of 128.
"""
import math

import numpy as np
import torch

own = False

C = float.fromhex("0x1.bb10f4p-8")   # codebook step, binary32
MULT = 0x9E3779B1


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# rows, cols: the coded matrix; transposed false: x has `rows` columns and y
# `cols`; true: the other way round (torch's [out, in] weights).
# slots: how tokens pick adapters: "one" (all the same), "each" (every token a
# request of its own, drawn, some without adapter), "prompts" (runs of tokens),
# "none" (no adapters).

def _lin(name, T, rows, cols, K, tr, dt, n, r, slots, wide=False):
    return dict(name=name, op="linear", T=T, rows=rows, cols=cols, K=K, transposed=tr, dtype=dt, n=n, r=r,
                slots=slots, wide=wide)


def _bwd(name, T, rows, cols, K, tr, dt, n, r, slots):
    return dict(_lin(name, T, rows, cols, K, tr, dt, n, r, slots), op="backward")


def _exp(name, T, E, rows, cols, K, tr, dt, skew):
    return dict(name=name, op="experts", T=T, E=E, rows=rows, cols=cols, K=K, transposed=tr, dtype=dt, skew=skew)


def listed():
    return [
        # one token of one request through a key projection: latency
        _lin("token_k_proj_k2", 1, 1024, 4096, 2, True, "bf16", 4, 16, "one"),
        # a few speculative tokens through a down projection, one bit, no adapters
        _lin("tokens7_down_k1", 7, 4096, 12288, 1, True, "fp16", 0, 0, "none"),
        # a decode batch of 64 requests, their adapters of mixed ranks, some without
        _lin("batch64_q_k3", 64, 4096, 4096, 3, False, "bf16", 40, 64, "each"),
        # short prompts and single tokens mixed, activations inside a wider buffer
        _lin("mixed333_gate_k4", 333, 12288, 4096, 4, True, "fp16", 6, 32, "prompts", True),
        # long prompts of several requests
        _lin("prompt4096_q_k2", 4096, 4096, 4096, 2, False, "bf16", 8, 16, "prompts"),
        # training adapters over frozen codes: a small, an odd and a large batch
        _bwd("grad96_k_k3", 96, 1024, 4096, 3, True, "fp16", 3, 8, "prompts"),
        _bwd("grad1001_o_k4", 1001, 4096, 4096, 4, False, "bf16", 5, 12, "each"),
        _bwd("grad4096_q_k2", 4096, 4096, 4096, 2, False, "bf16", 4, 64, "prompts"),
        # two tokens, two experts each: most experts have no row
        _exp("experts_4rows_k2", 4, 64, 2048, 1024, 2, False, "bf16", 0.0),
        # a decode batch over all experts
        _exp("experts_256rows_k3", 256, 64, 2048, 1024, 3, False, "fp16", 0.5),
        # input gradient (or the way back up) of ragged groups
        _exp("experts_3001rows_tr_k2", 3001, 64, 2048, 1024, 2, True, "bf16", 0.5),
        # a prompt's routed rows
        _exp("experts_16384rows_k4", 16384, 64, 2048, 1024, 4, False, "bf16", 0.5),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "experts"])
    K, tr, dt = rng.randint(1, 4), rng.random() < 0.5, rng.choice(["bf16", "fp16"])
    if op == "experts":
        E = rng.choice([5, 8, 16, 33, 64])
        rows, cols = 128 * _logint(rng, 4, 17), 128 * _logint(rng, 4, 17)
        T = _logint(rng, 1, 16384)
        while T * rows * cols > 16384 * 2048 * 1024 or E * rows * cols > 64 * 2048 * 1024:
            T, E, rows = max(1, T // 2), max(1, E // 2), max(512, 128 * (rows // 192))
        if rows == 24 * 128 or cols == 24 * 128:
            rows, cols = 25 * 128, 25 * 128
        return _strip(_exp("", T, E, rows, cols, K, tr, dt, rng.choice([0.0, 0.5, 0.9])))
    rows, cols = 128 * _logint(rng, 8, 96), 128 * _logint(rng, 8, 96)
    rows, cols = (3200 if v == 3072 else v for v in (rows, cols))
    T = _logint(rng, 1, 4096)
    n, r = _logint(rng, 1, 64), rng.randint(1, 64)
    while T * rows * cols > 4096 * 4096 * 4096 or rows * cols > 12288 * 4096:
        T, rows = max(1, T // 2), max(1024, 128 * (rows // 192))
    rows = 3200 if rows == 3072 else rows
    slots = rng.choice(["one", "each", "prompts"])
    if op == "linear":
        if rng.random() < 0.2:
            n, r, slots = 0, 0, "none"
        return _strip(_lin("", T, rows, cols, K, tr, dt, n, r, slots, rng.random() < 0.3))
    return _strip(_bwd("", T, rows, cols, K, tr, dt, n, r, slots))


def _strip(c):
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _dims(case):
    return (case["cols"], case["rows"]) if case["transposed"] else (case["rows"], case["cols"])


def _activations(g, T, n, dt, dev, wide=False):
    """Hidden states: rows of different magnitude, a few channels far above the rest."""
    x = torch.randn(T, n, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=dev))
    x[:, torch.randint(0, n, (max(1, n // 512),), generator=g, device=dev)] *= 20.0
    if wide:   # a column slice of a wider buffer, as behind a fused projection
        buf = torch.zeros(T, n + 192, dtype=dt, device=dev)
        buf[:, 64:64 + n] = x.to(dt)
        return buf[:, 64:64 + n]
    return x.to(dt)


def _coded(g, lead, rows, cols, K, dev):
    """A coded matrix as the quantizer leaves it: any code stream is a valid path;
    su signs, sv signs with the output channels' scales (a dead channel is 0)."""
    codes = torch.randint(-32768, 32768, (*lead, rows // 16, cols // 16, 16 * K), generator=g, device=dev,
                          dtype=torch.int32).to(torch.int16)
    su = (torch.randint(0, 2, (*lead, rows), generator=g, device=dev) * 2 - 1).float()
    sv = (torch.randint(0, 2, (*lead, cols), generator=g, device=dev) * 2 - 1).float()
    sv *= 0.02 * torch.exp(0.3 * torch.randn(*lead, cols, generator=g, device=dev))
    sv[..., cols // 3] = 0.0
    scale = 0.9 + 0.2 * torch.rand(lead if lead else (), generator=g, device=dev)
    return codes, su, sv, scale


def _slots(g, how, T, n, dev):
    if how == "one":
        return torch.full((T,), n // 2, dtype=torch.int32, device=dev)
    if how == "each":
        return torch.randint(-1, n, (T,), generator=g, device=dev, dtype=torch.int32)
    # runs: about two requests to an adapter, the first tokens without one
    cuts = torch.sort(torch.randint(0, T + 1, (2 * n,), generator=g, device=dev)).values
    run = torch.searchsorted(cuts, torch.arange(T, device=dev), right=True)
    which = torch.randint(0, n, (2 * n + 1,), generator=g, device=dev, dtype=torch.int32)
    which[0] = -1 if n > 1 else 0
    return which[run].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * seed + 17)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[case["dtype"]]
    T, rows, cols, K = case["T"], case["rows"], case["cols"], case["K"]
    n_in, n_out = _dims(case)
    s = dict(case=case, T=T, K=K, tr=bool(case["transposed"]), n_in=n_in, n_out=n_out, dt=dt)
    if case["op"] == "experts":
        E = case["E"]
        s["codes"], s["su"], s["sv"], s["scale"] = _coded(g, (E,), rows, cols, K, dev)
        # popularity of the experts: even, or a few taking most rows
        p = torch.rand(E, generator=g, device=dev) + 1e-3
        p = p ** (1.0 + 4.0 * case["skew"])
        pick = torch.multinomial(p / p.sum(), T, replacement=True, generator=g)
        counts = torch.bincount(pick, minlength=E)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), counts.cumsum(0)]).int()
        s["x"] = _activations(g, T, n_in, dt, dev)
        return s
    s["codes"], s["su"], s["sv"], s["scale"] = _coded(g, (), rows, cols, K, dev)
    s["x"] = _activations(g, T, n_in, dt, dev, case["wide"])
    n, r = case["n"], case["r"]
    if n:
        s["A"] = (torch.randn(n, r, n_in, generator=g, device=dev) / math.sqrt(n_in)).to(dt)
        s["B"] = (torch.randn(n, r, n_out, generator=g, device=dev) * 0.3).to(dt)
        s["gain"] = 0.25 + torch.rand(n, generator=g, device=dev)
        # a request's adapter has its own rank; its buffers are padded to r rows
        s["ranks"] = torch.randint(max(1, r // 4), r + 1, (n,), generator=g, device=dev, dtype=torch.int32)
        s["slots"] = _slots(g, case["slots"], T, n, dev)
    else:
        s["A"] = s["B"] = s["gain"] = s["ranks"] = s["slots"] = None
    if case["op"] == "backward":
        s["dy"] = (0.1 * torch.randn(T, n_out, generator=g, device=dev)).to(dt)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _hadamard(dev, dtype=torch.float32):
    i = torch.arange(128, device=dev)
    v = i[:, None] & i[None, :]
    for_bits = (v[..., None] >> torch.arange(7, device=dev)) & 1
    return (1 - 2 * (for_bits.sum(-1) & 1)).to(dtype)


def _weights(codes, su, sv, K, scale):
    """Codes [..., R, C, 16 K] -> W^ [..., 16 R, 16 C] in 32 bits."""
    dev = codes.device
    lead, (R, Cc, _) = codes.shape[:-3], codes.shape[-3:]
    w = codes.to(torch.int32) & 0xFFFF
    w = w.view(*lead, R, Cc, 8 * K, 2).flip(-1).reshape(*lead, R, Cc, 16 * K)       # stream order, 16 bits each
    p = ((torch.arange(256, device=dev) + 1) * K - 16) % (256 * K)                   # first bit of each window
    q = p // 16
    pair = (w[..., q].to(torch.int64) << 16) | w[..., (q + 1) % (16 * K)]
    x = ((pair >> (16 - p % 16)) & 0xFFFF) * MULT
    n = (x & 255) + ((x >> 8) & 255) + ((x >> 16) & 255) + ((x >> 24) & 255) - 510
    v = (n.float() * C).half().float()
    v = v.view(*lead, R, Cc, 16, 16).transpose(-3, -2).reshape(*lead, R // 8, 128, Cc * 16)
    H = _hadamard(dev)
    v = torch.matmul(H, v).reshape(*lead, R * 16, Cc // 8, 128)
    v = torch.matmul(v, H).reshape(*lead, R * 16, Cc * 16)
    return v * (su[..., :, None] * (scale * 2.0 ** -7)[..., None, None]) * sv[..., None, :]


def _pick(s):
    """[T, n r] factors: gain where the token uses this row of this adapter, else 0."""
    n, r = s["A"].shape[:2]
    dev = s["A"].device
    mine = s["slots"][:, None] == torch.arange(n, device=dev)
    row = torch.arange(r, device=dev)[None, :] < s["ranks"][:, None]
    return ((mine * s["gain"])[:, :, None] * row[None]).reshape(-1, n * r)


def _plain_linear(s):
    W = _weights(s["codes"], s["su"], s["sv"], s["K"], s["scale"])
    x = s["x"].float()
    y = x @ (W.t() if s["tr"] else W)
    if s["A"] is not None:
        A, B = s["A"].float().flatten(0, 1), s["B"].float().flatten(0, 1)
        y = y + ((x @ A.t()) * _pick(s)) @ B
    return y.to(s["dt"])


def _plain_backward(s):
    W = _weights(s["codes"], s["su"], s["sv"], s["K"], s["scale"])
    x, dy = s["x"].float(), s["dy"].float()
    A, B, f = s["A"].float().flatten(0, 1), s["B"].float().flatten(0, 1), _pick(s)
    g = (dy @ B.t()) * f
    dx = dy @ (W if s["tr"] else W.t()) + g @ A
    h = (x @ A.t()) * f
    return dict(dx=dx.to(s["dt"]), dA=(g.t() @ x).view(s["A"].shape).to(s["dt"]),
                dB=(h.t() @ dy).view(s["B"].shape).to(s["dt"]))


def _plain_experts(s):
    """Rows padded to the largest group, one batched product."""
    W = _weights(s["codes"], s["su"], s["sv"], s["K"], s["scale"])
    off = s["offsets"].long()
    count = off[1:] - off[:-1]
    cap = int(count.max())
    at = off[:-1, None] + torch.arange(cap, device=off.device)
    ok = torch.arange(cap, device=off.device) < count[:, None]
    x = s["x"].float()[torch.where(ok, at, 0)]
    y = torch.bmm(x, W.transpose(1, 2) if s["tr"] else W)
    out = torch.zeros(s["T"], s["n_out"], device=y.device)
    out[at[ok]] = y[ok]
    return out.to(s["dt"])


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"linear": _plain_linear, "backward": _plain_backward, "experts": _plain_experts}[op](s)
    import exl3_trellis_weight_gb300 as ex
    if op == "experts":
        return ex.expert_linear(s["x"], s["offsets"], s["codes"], s["su"], s["sv"], s["K"], s["scale"],
                                transposed=s["tr"])
    if op == "linear":
        return ex.linear(s["x"], s["codes"], s["su"], s["sv"], s["K"], s["scale"], transposed=s["tr"],
                         A=s["A"], B=s["B"], gain=s["gain"], slots=s["slots"], ranks=s["ranks"])
    return ex.linear_backward(s["dy"], s["x"], s["codes"], s["su"], s["sv"], s["K"], s["scale"],
                              transposed=s["tr"], A=s["A"], B=s["B"], gain=s["gain"], slots=s["slots"],
                              ranks=s["ranks"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    T, rows, cols, K = case["T"], case["rows"], case["cols"], case["K"]
    n_in, n_out = _dims(case)
    if case["op"] == "experts":
        used = case["E"] * (1.0 - (1.0 - 1.0 / case["E"]) ** T)    # experts with a row, about
        return dict(bytes=used * (rows * cols * K / 8 + 4 * (rows + cols)) + 2.0 * T * (n_in + n_out),
                    flops=2.0 * T * rows * cols)
    n, r = case["n"], 0.625 * case["r"]                            # mean rank of the drawn ones
    used = 0.0 if not n else 1.0 if case["slots"] == "one" else n * (1.0 - (1.0 - 1.0 / n) ** min(T, 2 * n)) if n > 1 else 1.0
    b = rows * cols * K / 8 + 4.0 * (rows + cols) + 2.0 * T * (n_in + n_out) + 2.0 * used * r * (n_in + n_out)
    f = 2.0 * T * rows * cols + (2.0 * T * r * (n_in + n_out) if n else 0.0)
    if case["op"] == "backward":
        b += 2.0 * T * n_in + 2.0 * n * case["r"] * (n_in + n_out)     # dx beside x and dy; dA and dB
        f += 4.0 * T * r * (n_in + n_out)
    return dict(bytes=b, flops=f)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _levels64(codes, K):
    """One coded matrix's levels V, bit by bit from the circular stream."""
    dev = codes.device
    R, Cc, _ = codes.shape
    j = torch.arange(256 * K, device=dev)
    word = (j // 16) ^ 1                                              # stored with neighbours swapped
    bits = (codes.long()[..., word] >> (15 - j % 16)) & 1
    state = torch.zeros(R, Cc, 256, dtype=torch.int64, device=dev)
    last = (torch.arange(256, device=dev) + 1) * K - 1
    for b in range(16):
        state += bits[..., (last - b) % (256 * K)] << b
    k = np.arange(65536, dtype=np.uint64) * np.uint64(MULT) % np.uint64(1 << 32)
    total = sum((k >> np.uint64(8 * b)) & np.uint64(255) for b in range(4)).astype(np.int64) - 510
    table = (total.astype(np.float32) * np.float32(C)).astype(np.float16).astype(np.float64)
    v = torch.from_numpy(table).to(dev)[state]
    return v.view(R, Cc, 16, 16).permute(0, 2, 1, 3).reshape(R * 16, Cc * 16)


def _turn64(m):
    """m [T, n] times the blockwise Sylvester matrix, by halves."""
    T, n = m.shape
    m = m.reshape(T * (n // 128), 128)
    for span in (1, 2, 4, 8, 16, 32, 64):
        m = m.reshape(-1, 128 // (2 * span), 2, span)
        m = torch.stack([m[:, :, 0] + m[:, :, 1], m[:, :, 0] - m[:, :, 1]], 2).reshape(-1, 128)
    return m.reshape(T, n)


def _apply64(x, codes, su, sv, K, scale, tr):
    V = _levels64(codes, K)
    left, right = (sv, su) if tr else (su, sv)
    z = _turn64(x * left.double()) @ (V.t() if tr else V)
    return _turn64(z) * right.double() * float(scale) / 128.0


def exact(case, seed):
    s = prepare(case, seed)
    x, K, tr = s["x"].double(), s["K"], s["tr"]
    if case["op"] == "experts":
        off = s["offsets"].tolist()
        y = torch.zeros(s["T"], s["n_out"], dtype=torch.float64, device=x.device)
        for e in range(case["E"]):
            if off[e + 1] > off[e]:
                y[off[e]:off[e + 1]] = _apply64(x[off[e]:off[e + 1]], s["codes"][e], s["su"][e], s["sv"][e], K,
                                                s["scale"][e], tr)
        return y
    args = (s["codes"], s["su"], s["sv"], K, s["scale"])
    if case["op"] == "linear":
        y = _apply64(x, *args, tr)
        for i in range(case["n"]):
            t, r = torch.nonzero(s["slots"] == i).flatten(), int(s["ranks"][i])
            h = float(s["gain"][i]) * (x[t] @ s["A"][i, :r].double().t())
            y[t] += h @ s["B"][i, :r].double()
        return y
    dy = s["dy"].double()
    dx = _apply64(dy, *args, not tr)
    dA, dB = torch.zeros_like(s["A"], dtype=torch.float64), torch.zeros_like(s["B"], dtype=torch.float64)
    for i in range(case["n"]):
        t, r, a = torch.nonzero(s["slots"] == i).flatten(), int(s["ranks"][i]), float(s["gain"][i])
        A, B = s["A"][i, :r].double(), s["B"][i, :r].double()
        g = a * (dy[t] @ B.t())
        dx[t] += g @ A
        dA[i, :r] = g.t() @ x[t]
        dB[i, :r] = a * (x[t] @ A.t()).t() @ dy[t]
    return dict(dx=dx, dA=dA, dB=dB)
