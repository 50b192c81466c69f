"""A coded layer in use: quantize weights, then serve and train on the codes.

Quantizes a projection and the weights of a few experts, and on the codes alone
  - decodes a batch of requests through the shared projection, each request with
    its own low-rank adapter (some without),
  - takes a training step of the adapters over the frozen codes,
  - sends the tokens through the experts that a router picked, and back.
Each result is compared with the same computation on the decoded weights.

  python examples/coded_layer.py            (needs the GPU; builds nothing)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exl3_trellis_weight_gb300 as ex  # noqa: E402
from exl3_trellis_weight_gb300 import inputs  # noqa: E402

DEV = torch.device("cuda:0")


def quantized(rows, cols, K, seed):
    """Codes, signs and scale of a random weight, and the decoded weight beside them."""
    W = inputs.linear_bf16(rows, cols, seed=seed, std=0.02).to(DEV)
    su, sv = (s.to(DEV) for s in inputs.sign_pair(rows, cols, seed))
    q = ex.quantize(W, su, sv, K, want_What=True)
    return q["codes"], su, sv, q["scale"], q["What"]


def close(got, want, what):
    err = float((got.double() - want.double()).norm() / want.double().norm())
    print(f"{what:42s} relative difference {err:.1e}")
    assert err < 1e-2, what


def main(hidden=512, out=256, tokens=24, adapters=3, rank=8, experts=4, K=2):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    codes, su, sv, scale, What = quantized(hidden, out, K, 11)
    x = torch.randn(tokens, hidden, generator=g, device=DEV).bfloat16()
    A = (torch.randn(adapters, rank, hidden, generator=g, device=DEV) / hidden ** 0.5).bfloat16()
    B = (torch.randn(adapters, rank, out, generator=g, device=DEV) * 0.1).bfloat16()
    gain = torch.full((adapters,), 2.0 / rank, device=DEV)
    slots = torch.randint(-1, adapters, (tokens,), generator=g, device=DEV, dtype=torch.int32)

    # a batch of requests through the shared projection
    kw = dict(A=A, B=B, gain=gain, slots=slots)
    y = ex.linear(x, codes, su, sv, K, scale, **kw)
    want = x.float() @ What
    for i in range(adapters):
        t = slots == i
        want[t] += gain[i] * (x[t].float() @ A[i].float().t()) @ B[i].float()
    close(y, want, "requests with adapters")

    # a training step of the adapters: the loss is half the squared result
    grad = ex.linear_backward(y, x, codes, su, sv, K, scale, **kw)
    t = slots == 0
    h = gain[0] * x[t].float() @ A[0].float().t()
    close(grad["dB"][0], h.t() @ y[t].float(), "gradient of the first adapter's B")
    B -= 0.01 * grad["dB"]
    A -= 0.01 * grad["dA"]

    # the tokens' experts: rows sorted by expert, weights never decoded in memory
    q = [quantized(hidden, out, K, 20 + e) for e in range(experts)]
    ecodes, esu, esv, escale, eW = (torch.stack(v) for v in zip(*q))
    pick = torch.randint(0, experts, (tokens,), generator=g, device=DEV)
    order = torch.argsort(pick, stable=True)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV),
                         torch.bincount(pick, minlength=experts).cumsum(0)]).int()
    xs = x[order]
    up = ex.expert_linear(xs, offsets, ecodes, esu, esv, K, escale)
    close(up, torch.einsum("tk,tkn->tn", xs.float(), eW[pick[order]]), "tokens through their experts")
    back = ex.expert_linear(up, offsets, ecodes, esu, esv, K, escale, transposed=True)
    close(back, torch.einsum("tn,tkn->tk", up.float(), eW[pick[order]]), "and their input gradient")
    torch.cuda.synchronize()
    assert ex.wait_timeouts() == 0


if __name__ == "__main__":
    main()
