"""Expert layers with many steps to a block: stages of inputs that are asked for again and again,
rings of codes that run on from tile to tile, sums handed over between whole tiles.

Tolerances are those of test_gpu_expert_layer.py, with one number of its own.  In float16 the
activations' two parts leave 2^-22 to rounding, and what counts are the matrix instructions'
sums: a set adds half of 2560 inputs in chains of 2560 / 128 / 2 steps of 8 tiles, each twice: 160
additions, which may cut what is below 2^-23 of the sum so far, half of that on average and
always the same way.  The sum so far is 0.71 of the last one in its root mean square:
160 * 2^-24 * 0.71 < 2^-17.  (The other product has a quarter of its 2048 inputs to a chain.)
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import oracle  # noqa: E402
from test_gpu_expert_layer import Experts, U, acts, gen, rms, within  # noqa: E402
from test_gpu_linear import DEV, weight64  # noqa: E402

E, H, F = 16, 2048, 2560
STAGES = 16                                # of any form, at most


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


def dense64(codes, su, sv, K, scale):
    """weight64 with its steps on the GPU (it takes a second for a matrix of this size)."""
    R, C, n = codes.shape
    w = (codes.view(R * C, 8 * K, 2).flip(2).reshape(R * C, n).long() & 0xFFFF)
    w = torch.cat([w[:, -1:], w, w[:, :1]], 1)                 # (a window of 16 bits may begin before the first)
    start = (torch.arange(256, device=DEV) + 1) * K            # in bits of w, which begins 16 before
    a, off = start // 16, start % 16
    state = (((w[:, a] << 16) | w[:, a + 1]) >> (16 - off)) & 0xFFFF
    table = torch.from_numpy(oracle.mul1_table().astype("float64")).to(DEV)
    V = table[state].view(R, C, 16, 16).permute(0, 2, 1, 3).reshape(R * 16, C * 16)
    Had = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    for _ in range(7):
        Had = torch.cat([torch.cat([Had, Had], 1), torch.cat([Had, -Had], 1)], 0)
    V = (Had @ V.reshape(R // 8, 128, C * 16)).view(R * 16, C * 16)
    V = (V.view(R * 16, C // 8, 128) @ Had).reshape(R * 16, C * 16)
    return V * su.double()[:, None] * sv.double()[None, :] * float(scale) / 128.0


class Large(Experts):
    def dense(self, e):
        if e not in self._dense:
            ms = [dense64(*(t[e] for t in m[:3]), K, m[3][e]) for m, K in ((self.gate, self.K), (self.up, self.K), (self.down, self.Kd))]
            self._dense[e] = [m.t() if self.tr else m for m in ms]
        return self._dense[e]


def expected(m, x, ids, weights, dt):
    y = torch.zeros(x.shape[0], m.H, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(y)
    r = 2.0 ** -11 / math.sqrt(3) if dt == "bf16" else 2.0 ** -17
    for e in range(m.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        G, Up, D = m.dense(e)
        xe, w = x[t].double(), weights[t, j].double()[:, None]
        a, b = xe @ G, xe @ Up
        s = a * torch.sigmoid(a)
        dh = 1.1 * b.abs() * r * rms(a, m.right(m.gate, e)) + s.abs() * r * rms(b, m.right(m.up, e))
        left = m.left(m.down, e)
        q = (dh * left).norm(dim=1, keepdim=True) / (s * b * left).norm(dim=1, keepdim=True).clamp_min(1e-300)
        P = w * (s * b @ D)
        y.index_add_(0, t, P)
        tol.index_add_(0, t, 6 * (r + q) * rms(P, m.right(m.down, e)) + 2.0 ** -16 * P.abs())
    return y, tol + U[dt] * y.abs() * (1 + 2.0 ** -10) + 2.0 ** -25


def tile_rows(T, top_k, dt):
    """Rows of a tile, as the library chooses them."""
    n = T * top_k
    return 8 if T <= 8 or n <= 4 * E else 16 if T <= 16 or dt == "fp16" or n <= 10 * E else 32


def test_the_decoder_of_these_tests(ex):
    g = gen(1)
    for K in (1, 2, 3, 4):
        m = Experts(g, 1, 128, 256, K, K, False)
        t = [v[0] for v in m.gate]
        assert torch.equal(dense64(*t[:3], K, t[3]), weight64(*t[:3], K, t[3]))


@pytest.mark.parametrize("K,Kd", [(1, 2), (2, 3), (3, 4), (4, 1), (4, 4)])
@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_many_steps_a_block(ex, K, Kd, tr, dt):
    g = gen(K + 10 * Kd)
    m = Large(g, E, H, F, K, Kd, tr)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seen = set()
    for T, top_k in ((8, 16), (16, 16), (61, 8), (200, 8)):
        x, w = acts(g, T, H, dt), torch.rand(T, top_k, generator=g, device=DEV) / top_k
        ids = torch.randint(-1, E, (T, top_k), generator=g, device=DEV, dtype=torch.int32)
        if top_k == E:
            ids[:] = torch.arange(E, device=DEV)
            ids[T // 2, 3] = -1
        rows = tile_rows(T, top_k, dt)
        seen.add(rows)
        tiles = sum(-(-int(c) // rows) for c in torch.bincount(ids[ids >= 0], minlength=E))
        assert tiles * (H // 128) * (F // 128) // sms >= 2 * STAGES
        y = m.run(ex, x, top_k, ids=ids, weights=w)
        within(y, expected(m, x, ids, w, dt))
        for _ in range(5):
            assert torch.equal(m.run(ex, x, top_k, ids=ids, weights=w), y)
    assert seen == ({8, 16, 32} if dt == "bf16" else {8, 16})
