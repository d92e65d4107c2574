"""The router and the experts' products on the GPU against their definitions in 64 bits
(tests/experts_oracle.py, which derives the bounds)."""
import math

import pytest
import torch

import experts_oracle as eo
import ffn_oracle as fo
from test_ffn_gpu import BF16, F16, Band, gen, lm, near, rand, say, strided  # noqa: F401

pytestmark = pytest.mark.gpu
F32 = torch.float32


# ---- router ---------------------------------------------------------------------------

# M, E, k, groups, top_groups, best
ROUTES = [(1, 1, 1, 1, 1, 1), (1, 64, 8, 1, 1, 1), (3, 2, 2, 1, 1, 1), (7, 10, 3, 5, 2, 2),
          (65, 63, 6, 1, 1, 1), (33, 65, 8, 1, 1, 1), (130, 120, 6, 8, 3, 1), (50, 256, 8, 8, 4, 2),
          (20, 257, 8, 1, 1, 1), (9, 512, 64, 64, 16, 2), (6, 1000, 16, 4, 1, 2),
          (5, 1024, 64, 16, 16, 1), (40, 8, 8, 8, 8, 2), (12, 12, 4, 3, 1, 2)]


def logits_of(g, M, E, dtype):
    """Normal logits among which some rows have masked experts, ties, infinities and NaN."""
    x = torch.randn((M, E), generator=g, device="cuda") * 2
    for i in range(M):
        kind = i % 9
        if kind == 1:
            x[i] = -math.inf
        elif kind == 2:
            x[i, 1:] = -math.inf
        elif kind == 3:
            x[i, ::2] = math.nan
        elif kind == 4:
            x[i] = torch.round(x[i])
        elif kind == 5:
            x[i, E // 2] = math.inf
            x[i, E - 1] = math.inf
        elif kind == 6:
            x[i] = torch.finfo(dtype).min
        elif kind == 7:
            x[i] = x[i] * 30 - 50
    return x.to(dtype)


@pytest.mark.parametrize("M,E,k,groups,top_groups,best", ROUTES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_route(lm, M, E, k, groups, top_groups, best, scores, renorm, dtype):
    say("route", M, E, k, groups, scores, renorm, dtype)
    g = gen(M + E + k)
    x = logits_of(g, M, E, dtype)
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda") if (M + E) % 2 else None
    kw = dict(scores=scores, renormalize=renorm, scale=2.5)
    ids, w = lm.llmint8_route(strided(x), k, bias=bias, groups=groups, top_groups=top_groups,
                              group_best=best, **kw)
    want = eo.choose(x, k, scores, bias, groups, top_groups, best)
    # a value that underflows, or two saturated ones, is a tie in 64 bits: the same rule there
    assert torch.equal(ids, want)
    y, tol = eo.mix(x, ids, scores, renorm)
    near(w, (2.5 * y, 2.5 * tol + 2 * eo.EPS * y))
    assert bool((w[ids < 0] == 0).all())
    d = torch.randn((M, k), generator=g, device="cuda")
    dx, tol = eo.route_backward(d, x, ids, scores, renorm, 2.5)
    if dtype is not F32:
        tol = fo.stored(dx, tol, dtype)
    out = Band(M, E, dtype)
    lm.llmint8_route_backward(d, strided(x), ids, dlogits=out.t, **kw)
    out.check()
    near(out.t, (dx, tol))
    again = lm.llmint8_route_backward(d, x, ids, **kw)
    assert torch.equal(again.view(torch.uint8), out.t.contiguous().view(torch.uint8))


def test_route_backward_of_an_expert_named_twice_and_of_none(lm):
    say("route backward, ids given")
    g = gen(2)
    x = torch.randn((4, 10), generator=g, device="cuda")
    ids = torch.tensor([[3, 3, 9], [-1, 2, 2], [0, 10, 1], [-7, -1, -1]], dtype=torch.int32,
                       device="cuda")
    d = torch.randn((4, 3), generator=g, device="cuda")
    for scores in ("softmax", "sigmoid"):
        for renorm in (False, True):
            near(lm.llmint8_route_backward(d, x, ids, scores=scores, renormalize=renorm),
                 eo.route_backward(d, x, ids, scores, renorm, 1.0))


@pytest.mark.parametrize("M,k,E", [(1, 1, 1), (1, 8, 64), (5, 3, 7), (333, 3, 11), (1000, 8, 256),
                                   (4097, 2, 3), (700, 64, 1024), (8192, 1, 4), (9000, 8, 40),
                                   (70001, 2, 5)])
def test_plan(lm, M, k, E):
    say("plan", M, k, E)
    g = gen(M + k + E)
    ids = torch.randint(-1, E + 1, (M, k), generator=g, device="cuda", dtype=torch.int32)
    if M == 5:
        ids[:] = -1
    if M == 8192:
        ids[:] = 2
    got = lm.llmint8_expert_plan(ids, E)
    for name, a, b in zip(got._fields, got, eo.plan(ids, E)):
        assert torch.equal(a, b), name


# ---- experts' products ----------------------------------------------------------------

# M, K, N, E, k, masked: single tokens; few rows of 16, 32 and 64 a group; 128-tiles; 256-tiles
# whose last one has less and more than half of its rows; one expert; experts without rows
EXPERTS = [(1, 8, 8, 1, 1, 0.0), (1, 1040, 520, 64, 8, 0.0), (1, 4096, 136, 3, 1, 0.0),
           (2, 72, 1032, 16, 2, 0.0), (7, 264, 24, 5, 5, 0.5), (40, 1000, 72, 4, 2, 0.1),
           (96, 520, 264, 12, 4, 0.0), (100, 64, 1032, 4, 1, 0.1), (333, 1040, 520, 11, 3, 0.05),
           (130, 264, 136, 1, 1, 0.0), (600, 72, 520, 4, 1, 0.0), (1000, 264, 392, 6, 2, 0.1),
           (2000, 136, 72, 3, 2, 0.0), (515, 2056, 264, 2, 2, 0.0), (64, 2048, 2056, 40, 6, 0.2),
           (300, 264, 4104, 2, 1, 0.0)]


def pad3(t):
    """t [E, rows, cols] in a larger buffer with NaN between rows and between experts."""
    E, r, c = t.shape
    big = torch.full((E, r + 3, c + 16), float("nan"), dtype=t.dtype, device=t.device)
    big[:, :r, :c] = t
    return big[:, :r, :c]


def ids_of(g, M, E, k, masked):
    x = 1.5 * torch.randn((M, E), generator=g, device="cuda")
    x += 1.5 * torch.randn((1, E), generator=g, device="cuda")
    ids = x.argsort(1, descending=True)[:, :k].to(torch.int32).contiguous()
    ids[torch.rand((M, k), generator=g, device="cuda") < masked] = -1
    return ids


def rounded(lm, M, K, N, E, k):
    """Whether the second product's rows go through 16 bits before they are summed (with few rows
    an expert they stay in fp32, and the workspace is of that size, in multiples of 256 bytes)."""
    return lm.llmint8_experts_matmul_workspace_size(M, K, N, E, k) <= -(-M * k * K * 2 // 256) * 256


class Experts:
    def __init__(self, lm, M, K, N, E, k, masked, dtype, seed=0):
        g = gen(M + 3 * K + 5 * N + E + seed)
        self.ids = ids_of(g, M, E, k, masked)
        self.plan = lm.llmint8_expert_plan(self.ids, E)
        self.p = eo.plan(self.ids, E)
        self.last = int(self.p[0][-1])
        self.w = torch.rand((M, k), generator=g, device="cuda") * 2 - 0.5
        self.X = rand(g, M, K, dtype)
        self.Wg, self.Wu, self.Wd = (
            rand(g, E * a, b, dtype, 0.05).view(E, a, b) for a, b in ((K, N), (K, N), (N, K)))
        R = M * k
        self.H, self.dH = rand(g, R, N, dtype), rand(g, R, N, dtype, 0.5)
        self.G, self.U = rand(g, R, N, dtype, 1.5), rand(g, R, N, dtype, 1.5)
        self.R, self.dY = rand(g, M, K, dtype), rand(g, M, K, dtype, 0.5)
        self.name = fo.ACTS[1 + (M + K + N) // 8 % 4]
        self.rounded = rounded(lm, M, K, N, E, k)


def rows_only(got, want, last):
    near(got[:last], tuple(t[:last] for t in want))


@pytest.mark.parametrize("M,K,N,E,k,masked", EXPERTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_experts_forward(lm, M, K, N, E, k, masked, dtype):
    say("experts forward", M, K, N, E, k, dtype)
    s = Experts(lm, M, K, N, E, k, masked, dtype)
    H = Band(M * k, N, dtype)
    before = H.t.clone()
    h, G, U = lm.llmint8_experts_gated(strided(s.X), pad3(s.Wg), pad3(s.Wu), s.plan, weights=s.w,
                                       activation=s.name, save="full", H=H.t)
    assert h is H.t
    H.check()
    want = eo.gated(s.X.double(), s.Wg.double(), s.Wu.double(), s.p, s.w, s.name, dtype)
    for name, t in (("H", h), ("G", G), ("U", U)):
        rows_only(t, want[name], s.last)
    assert torch.equal(h[s.last:], before[s.last:]), "wrote behind the last row"
    # contiguous, without saving or weights, twice the same
    a = lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, s.plan, activation=s.name)
    b = lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, s.plan, activation=s.name)
    assert torch.equal(a[:s.last], b[:s.last])
    rows_only(a, eo.gated(s.X.double(), s.Wg.double(), s.Wu.double(), s.p, None, s.name, dtype)["H"],
              s.last)
    # rows that no plan names hold NaN: nothing reads them
    Hn = s.H.clone()
    Hn[s.last:] = math.nan
    Y = Band(M, K, dtype)
    lm.llmint8_experts_matmul(strided(Hn), pad3(s.Wd), s.plan, residual=strided(s.R), Y=Y.t)
    Y.check()
    near(Y.t, eo.matmul(s.H.double(), s.Wd.double(), s.p, s.R.double(), dtype, s.rounded))
    near(lm.llmint8_experts_matmul(Hn, s.Wd, s.plan),
         eo.matmul(s.H.double(), s.Wd.double(), s.p, None, dtype, s.rounded))


@pytest.mark.parametrize("M,K,N,E,k,masked", EXPERTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_experts_backward(lm, M, K, N, E, k, masked, dtype):
    say("experts backward", M, K, N, E, k, dtype)
    s = Experts(lm, M, K, N, E, k, masked, dtype, seed=1)
    for t in (s.H, s.dH, s.G, s.U):
        t[s.last:] = math.nan
    z = [t.clone() for t in (s.H, s.dH, s.G, s.U)]
    for t in z:
        t[s.last:] = 0
    H0, dH0, G0, U0 = (t.double() for t in z)
    dH = Band(M * k, N, dtype)
    before = dH.t.clone()
    dWd = pad3(torch.zeros_like(s.Wd))
    lm.llmint8_experts_matmul_backward(strided(s.dY), strided(s.H), pad3(s.Wd), s.plan, dH=dH.t,
                                       dWd=dWd)
    dH.check()
    assert torch.equal(dH.t[s.last:], before[s.last:]), "wrote behind the last row"
    want = eo.matmul_backward(s.dY.double(), H0, s.Wd.double(), s.p, dtype)
    rows_only(dH.t, want["dH"], s.last)
    near(dWd, want["dWd"])
    only = lm.llmint8_experts_matmul_backward(s.dY, None, s.Wd, s.plan, need_dW=False)
    assert only[1] is None and torch.equal(only[0][:s.last], dH.t[:s.last])
    only = lm.llmint8_experts_matmul_backward(s.dY, s.H, s.Wd, s.plan, need_dH=False)
    assert only[0] is None and torch.equal(only[1], dWd)

    dX = Band(M, K, dtype)
    dWg, dWu = pad3(torch.zeros_like(s.Wg)), pad3(torch.zeros_like(s.Wu))
    out = lm.llmint8_experts_gated_backward(strided(s.dH), strided(s.X), pad3(s.Wg), pad3(s.Wu),
                                            strided(s.G), strided(s.U), s.plan, weights=s.w,
                                            activation=s.name, dX=dX.t, dWg=dWg, dWu=dWu)
    dX.check()
    want = eo.gated_backward(dH0, s.X.double(), s.Wg.double(), s.Wu.double(), G0, U0, s.p, s.w,
                             s.name, dtype)
    for name, t in zip(("dX", "dWg", "dWu", "dw"), out):
        near(t, want[name])
    only = lm.llmint8_experts_gated_backward(s.dH, None, s.Wg, s.Wu, s.G, s.U, s.plan, weights=s.w,
                                             activation=s.name, need_dW=False, need_dweights=False)
    assert only[1] is only[2] is only[3] is None and torch.equal(only[0], dX.t)
    only = lm.llmint8_experts_gated_backward(s.dH, s.X, s.Wg, s.Wu, s.G, s.U, s.plan,
                                             activation=s.name, need_dX=False)
    want = eo.gated_backward(dH0, s.X.double(), s.Wg.double(), s.Wu.double(), G0, U0, s.p, None,
                             s.name, dtype)
    assert only[0] is None
    for name, t in zip(("dWg", "dWu", "dw"), only[1:]):
        near(t, want[name])
