"""The routed operators and the block-scaled FP8 product as a user calls them: together, on
another stream, two at once, in a captured and replayed graph, at sizes past 2 GiB and 2^32
elements, with plans that no ids give, the same expert twice, broadcast weights, and entries
that are not finite."""
import math

import pytest
import torch

import experts_oracle as eo
import ffn_oracle as fo
import fp8_block_oracle as bo
import test_experts_gpu as base
import test_fp8_block_gpu as fp8
from test_experts_gpu import Experts, ids_of, rows_only
from test_ffn_gpu import BF16, F16, Band, gen, lm, near, rand, say  # noqa: F401

pytestmark = pytest.mark.gpu

# M, K, N, E, k, masked: kernel variants that the lists of test_experts_gpu.py and
# test_fp8_block_gpu.py do not reach, and tiles of 256 with odd sizes on every side
EXPERTS = [(362, 2384, 8, 62, 2, 0.0), (2038, 2272, 8, 42, 1, 0.0), (202, 8, 72, 165, 1, 0.0),
           (204, 8, 136, 97, 6, 0.1), (27, 10312, 240, 17, 5, 0.0), (3902, 8, 80, 227, 1, 0.0),
           (2951, 8, 1344, 118, 1, 0.0), (35, 144, 8, 122, 4, 0.0), (162, 72, 1056, 102, 7, 0.0),
           (362, 72, 1064, 123, 6, 0.0), (7187, 136, 88, 53, 8, 0.0), (14501, 8, 472, 8, 7, 0.0),
           (16262, 400, 8, 19, 7, 0.0), (6001, 520, 1032, 24, 4, 0.1)]
FP8 = [(7107, 2016, 8), (553, 16, 26760), (129, 10480, 5600), (1, 2080, 8), (3, 6416, 5800)]


@pytest.mark.parametrize("M,K,N,E,k,masked", EXPERTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_experts_variants(lm, M, K, N, E, k, masked, dtype):
    base.test_experts_forward(lm, M, K, N, E, k, masked, dtype)
    torch.cuda.empty_cache()
    base.test_experts_backward(lm, M, K, N, E, k, masked, dtype)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,k,E", [(5, 3, 7), (999, 7, 40), (24576, 1, 3), (24577, 1, 3), (4100, 8, 1024), (12099, 3, 257),
                                   (40000, 8, 1024), (300001, 1, 7), (262144, 1, 1),
                                   (131073, 64, 65)])
def test_plans_of_many_pairs(lm, M, k, E):
    """One launch, and chunks of 1024 pairs and of more, against a stable sort by expert."""
    say("plan", M, k, E)
    g = gen(M)
    ids = torch.randint(-2, E + 2, (M, k), generator=g, device="cuda", dtype=torch.int32)
    ids[M // 3:M // 2] = E // 2  # long runs of one expert
    key = torch.where((ids < 0) | (ids >= E), E, ids).reshape(-1).cpu().long()
    order = torch.sort(key, stable=True).indices
    last = int((key < E).sum())
    places = torch.empty_like(order)
    places[order] = torch.arange(order.numel())
    places[key == E] = -1
    order[last:] = -1
    offsets = torch.searchsorted(key.sort().values, torch.arange(E + 1))
    apart = torch.empty((M * k + 1,), dtype=torch.int32, device="cuda")[1:].view(M, k)
    for given in (ids, ids, apart.copy_(ids)):  # the last 4 bytes past a multiple of 16
        got = lm.llmint8_expert_plan(given, E)
        assert torch.equal(got.offsets.cpu().long(), offsets)
        assert torch.equal(got.order.cpu().long(), order)
        assert torch.equal(got.places.cpu().long(), places.view(M, k))


@pytest.mark.parametrize("E,k,groups,top,best", [(256, 8, 8, 4, 2), (256, 8, 1, 1, 1), (64, 6, 4, 2, 1),
                                                 (512, 16, 16, 5, 2), (1000, 3, 1, 1, 1)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_choices_between_close_values(lm, E, k, groups, top, best, scores):
    """Scores with a bias that differ by fractions of what fp32 can tell: the choice is that of 64
    bits. Rows of logits a few units of their last place apart, whose biases make up for most
    of it; tiny scores beside a bias of 1; ties; and rows with one clear order."""
    say("close values", E, k, groups, scores)
    g = gen(E + k)
    M = 96
    base = torch.randn((M, 1), generator=g, device="cuda")
    x = base + torch.randint(-3, 4, (M, E), generator=g, device="cuda") * 2.0 ** -22
    x[24:48] = torch.randn((24, E), generator=g, device="cuda") - 60
    x[48:60] = torch.randn((12, E), generator=g, device="cuda") * 3
    x[60:72, ::2] = x[60:72, 1::2]
    x[72:84] = torch.randn((12, E), generator=g, device="cuda").to(BF16).float()
    bias = torch.randint(-2, 3, (E,), generator=g, device="cuda") * 2.0 ** -26
    for b in (bias, bias + 1, torch.zeros_like(bias)):
        kw = dict(scores=scores, bias=b, groups=groups, top_groups=top, group_best=best)
        ids, w = lm.llmint8_route(x, k, **kw)
        assert torch.equal(ids, eo.choose(x, k, scores, b, groups, top, best))
        near(w, eo.mix(x, ids, scores, False))


@pytest.mark.parametrize("M,K,N", FP8)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_fp8_variants(lm, M, K, N, dtype):
    fp8.test_linear(lm, M, K, N, dtype)


class Layer:
    """A routed block with a residual, forward and backward, from the router's logits on."""

    def __init__(self, lm, M, K, N, E, k, dtype, seed=0):
        g = gen(seed + M + K)
        self.lm, self.k, self.E = lm, k, E
        self.X, self.D = rand(g, M, K, dtype), rand(g, M, K, dtype, 0.5)
        self.logits = torch.randn((M, E), generator=g, device="cuda") * 1.5
        self.Wg, self.Wu, self.Wd = (rand(g, E * a, b, dtype, 0.3 / math.sqrt(a) * 3).view(E, a, b)
                                     for a, b in ((K, N), (K, N), (N, K)))
        self.how = dict(scores="sigmoid", renormalize=True, scale=1.5)

    def step(self):
        lm = self.lm
        ids, w = lm.llmint8_route(self.logits, self.k, **self.how)
        plan = lm.llmint8_expert_plan(ids, self.E)
        H, G, U = lm.llmint8_experts_gated(self.X, self.Wg, self.Wu, plan, weights=w, save="full")
        Y = lm.llmint8_experts_matmul(H, self.Wd, plan, residual=self.X)
        dH, dWd = lm.llmint8_experts_matmul_backward(self.D, H, self.Wd, plan)
        dX, dWg, dWu, dw = lm.llmint8_experts_gated_backward(
            dH, self.X, self.Wg, self.Wu, G, U, plan, weights=w)
        dlogits = lm.llmint8_route_backward(dw, self.logits, ids, **self.how)
        self.held = dict(ids=ids, w=w, plan=plan, H=H, G=G, U=U, Y=Y, dH=dH, dWd=dWd, dX=dX,
                         dWg=dWg, dWu=dWu, dw=dw, dlogits=dlogits)
        return [ids, w, Y, dWd, dX, dWg, dWu, dw, dlogits]


SIZES = [(1, 256, 136, 8, 2), (45, 264, 520, 12, 3), (700, 264, 136, 4, 2)]


@pytest.mark.parametrize("M,K,N,E,k", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_layer(lm, M, K, N, E, k, dtype):
    """Every step of a layer against 64 bits, from what the step before gave."""
    say("layer", M, K, N, E, k, dtype)
    a = Layer(lm, M, K, N, E, k, dtype)
    a.step()
    h, d = a.held, lambda t: t.double()  # noqa: E731
    assert torch.equal(h["ids"], eo.choose(a.logits, k, "sigmoid"))
    y, tol = eo.mix(a.logits, h["ids"], "sigmoid", True)
    near(h["w"], (1.5 * y, 1.5 * tol + 2 * eo.EPS * y))
    p = eo.plan(h["ids"], E)
    for got, want in zip(h["plan"], p):
        assert torch.equal(got, want)
    want = eo.gated(d(a.X), d(a.Wg), d(a.Wu), p, h["w"], "silu", dtype)
    for n in "HGU":
        near(h[n], want[n])
    rounded = base.rounded(lm, M, K, N, E, k)
    near(h["Y"], eo.matmul(d(h["H"]), d(a.Wd), p, d(a.X), dtype, rounded))
    want = eo.matmul_backward(d(a.D), d(h["H"]), d(a.Wd), p, dtype)
    near(h["dH"], want["dH"]), near(h["dWd"], want["dWd"])
    want = eo.gated_backward(d(h["dH"]), d(a.X), d(a.Wg), d(a.Wu), d(h["G"]), d(h["U"]), p, h["w"],
                             "silu", dtype)
    near(h["dX"], want["dX"]), near(h["dWg"], want["dWg"]), near(h["dWu"], want["dWu"])
    near(h["dw"], want["dw"])
    near(h["dlogits"], eo.route_backward(h["dw"], a.logits, h["ids"], "sigmoid", True, 1.5))


@pytest.mark.parametrize("M,K,N,E,k", SIZES)
def test_gradients_against_differences(lm, M, K, N, E, k):
    """The layer's gradients against central differences of its output in 64 bits, with the
    choice held, along random directions. A gradient's entries have independent errors: the
    roundings of H, G, U, dH, dG, dU and of itself, below 8 u of its norm in all; that of a
    logit sums products of twice w dw, which cancel, so its errors are measured by them."""
    say("differences", M, K, N, E, k)
    a = Layer(lm, M, K, N, E, k, F16, seed=3)
    a.step()
    h = a.held
    ids = h["ids"].long()
    D, tok = a.D.double(), torch.arange(M, device="cuda")

    def loss(x, wg, wu, wd, logits):
        s = torch.sigmoid(torch.gather(logits, 1, ids))
        w = 1.5 * s / s.sum(1, keepdim=True)
        total = x.new_zeros(())
        for j in range(k):
            for e in range(E):
                t = tok[ids[:, j] == e]
                if len(t):
                    hid = fo.act("silu", x[t] @ wg[e]) * (x[t] @ wu[e]) * w[t, j, None]
                    total = total + (D[t] * (hid @ wd[e])).sum()
        return total
    at = [t.double() for t in (a.X, a.Wg, a.Wu, a.Wd, a.logits)]
    g = gen(8)
    for i, name in enumerate(("dX", "dWg", "dWu", "dWd", "dlogits")):
        grad = h[name].double()
        V = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        V /= V.norm()
        step = 1e-4
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * V, at[i] - step * V
        want = float((loss(*up) - loss(*down)) / (2 * step))
        got = float((grad * V).sum())
        size = float(grad.norm())
        if name == "dlogits":
            size = 2 * float((h["w"] * h["dw"]).double().norm())
        assert abs(got - want) <= 8 * fo.U[F16] * size + 1e-6, (name, got, want)


def test_other_stream_and_two_at_once(lm):
    say("streams")
    a, b = Layer(lm, 45, 264, 520, 12, 3, F16), Layer(lm, 700, 264, 136, 4, 2, BF16, seed=1)
    want = [[t.clone() for t in x.step()] for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(x.step())
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for t, w in zip(run, want[i]):
                assert torch.equal(t, w)


@pytest.mark.parametrize("M,K,N,E,k", SIZES + [(3000, 264, 136, 40, 8)])
def test_graph_replay(lm, M, K, N, E, k):
    """The captured step follows its inputs: new logits, so other experts, in every replay."""
    say("graph replay", M, K, N, E, k)
    a = Layer(lm, M, K, N, E, k, BF16, seed=2)
    g = gen(5)
    wq, sw = lm.llmint8_quantize_blockwise_fp8(rand(g, K // 16 * 16, 264, BF16, 0.1))
    x8 = rand(g, M, K // 16 * 16, BF16)

    def step():
        return [*a.step(), lm.llmint8_linear_blockwise_fp8(x8, wq, sw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        a.logits.copy_(torch.randn((M, E), generator=g, device="cuda"))
        if rep == 2:
            a.logits[:] = -math.inf  # no rows at all
        a.X.copy_(rand(g, M, K, BF16))
        x8.copy_(rand(g, M, K // 16 * 16, BF16))
        want = [t.clone() for t in step()]  # eager work between replays
        for t in out:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, w) in enumerate(zip(out, want)):
            assert torch.equal(t, w), (rep, i)


@pytest.mark.parametrize("M,K,N,E,k", SIZES + [(2000, 264, 1032, 4, 4)])
def test_no_rows_and_one_expert_for_all(lm, M, K, N, E, k):
    say("no rows", M, K, N, E, k)
    s = Experts(lm, M, K, N, E, k, 0.0, F16)
    none = torch.full((M, k), -1, dtype=torch.int32, device="cuda")
    plan = lm.llmint8_expert_plan(none, E)
    H = Band(M * k, N, F16)
    before = H.t.clone()
    lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, plan, weights=s.w, H=H.t)
    H.check()
    assert torch.equal(H.t, before)
    assert torch.equal(lm.llmint8_experts_matmul(s.H, s.Wd, plan, residual=s.R), s.R)
    assert not bool(lm.llmint8_experts_matmul(s.H, s.Wd, plan).any())
    dH = before.clone()
    _, dWd = lm.llmint8_experts_matmul_backward(s.dY, s.H, s.Wd, plan, dH=dH)
    assert torch.equal(dH, before) and not bool(dWd.any())
    for t in lm.llmint8_experts_gated_backward(s.dH, s.X, s.Wg, s.Wu, s.G, s.U, plan, weights=s.w):
        assert not bool(t.any())
    # all tokens' first choice is the last expert, their others none
    none[:, 0] = E - 1
    plan, p = lm.llmint8_expert_plan(none, E), eo.plan(none, E)
    h = lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, plan, weights=s.w)
    rows_only(h, eo.gated(s.X.double(), s.Wg.double(), s.Wu.double(), p, s.w, "silu", F16)["H"], M)
    near(lm.llmint8_experts_matmul(s.H, s.Wd, plan, residual=s.R),
         eo.matmul(s.H.double(), s.Wd.double(), p, s.R.double(), F16, s.rounded))


@pytest.mark.parametrize("M,K,N,E,k", [(40, 264, 136, 6, 4), (900, 136, 264, 3, 3)])
def test_an_expert_named_twice(lm, M, K, N, E, k):
    say("expert twice", M, K, N, E, k)
    s = Experts(lm, M, K, N, E, k, 0.0, BF16)
    s.ids[:, 1] = s.ids[:, 0]
    s.ids[::3, 2] = s.ids[::3, 0]
    plan, p = lm.llmint8_expert_plan(s.ids, E), eo.plan(s.ids, E)
    near(lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, plan, weights=s.w),
         eo.gated(s.X.double(), s.Wg.double(), s.Wu.double(), p, s.w, "silu", BF16)["H"])
    near(lm.llmint8_experts_matmul(s.H, s.Wd, plan, residual=s.R),
         eo.matmul(s.H.double(), s.Wd.double(), p, s.R.double(), BF16, s.rounded))
    got = lm.llmint8_experts_gated_backward(s.dH, s.X, s.Wg, s.Wu, s.G, s.U, plan, weights=s.w)
    want = eo.gated_backward(s.dH.double(), s.X.double(), s.Wg.double(), s.Wu.double(),
                             s.G.double(), s.U.double(), p, s.w, "silu", BF16)
    for t, n in zip(got, ("dX", "dWg", "dWu", "dw")):
        near(t, want[n])


@pytest.mark.parametrize("M,K,N,E,k", [(1, 264, 136, 6, 4), (300, 136, 264, 30, 3),
                                       (3000, 136, 264, 5, 3)])
@pytest.mark.parametrize("kind", range(4))
def test_plans_that_no_ids_give(lm, M, K, N, E, k, kind):
    """Offsets, order and places of any value: the results are of no use, and nothing outside
    the outputs is written. (What is read from a plan is checked against the buffers' rows.)"""
    say("wrong plans", M, K, N, E, k, kind)
    g = gen(kind)
    s = Experts(lm, M, K, N, E, k, 0.0, F16)
    R = M * k
    far = lambda *n: torch.randint(-2 ** 31, 2 ** 31 - 1, n, generator=g, device="cuda",  # noqa: E731
                                   dtype=torch.int32)
    some = lambda *n: torch.randint(-3, R + 3, n, generator=g, device="cuda",  # noqa: E731
                                    dtype=torch.int32)
    if kind == 0:
        plan = lm.ExpertPlan(far(E + 1), far(R), far(M, k))
    elif kind == 1:
        plan = lm.ExpertPlan(some(E + 1), some(R), some(M, k))
    elif kind == 2:
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1::2] = R  # every other expert has all rows
        plan = lm.ExpertPlan(offsets, s.plan.order, s.plan.places)
    else:  # the plan of other experts
        ids = ids_of(g, M, E, k, 0.5)
        other = lm.llmint8_expert_plan(ids, E)
        plan = lm.ExpertPlan(other.offsets, s.plan.order, other.places)
    H, Y, dH, dX = Band(R, N, F16), Band(M, K, F16), Band(R, N, F16), Band(M, K, F16)
    dW = torch.full((E + 2, K, N), 7.0, dtype=F16, device="cuda")
    dV, dD = dW.clone(), torch.full((E + 2, N, K), 7.0, dtype=F16, device="cuda")
    dw = Band(M, k, torch.float32, pad=0)
    lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, plan, weights=s.w, H=H.t, save="full")
    lm.llmint8_experts_matmul(s.H, s.Wd, plan, Y=Y.t)
    lm.llmint8_experts_matmul_backward(s.dY, s.H, s.Wd, plan, dH=dH.t, dWd=dD[1:E + 1])
    lm.llmint8_experts_gated_backward(s.dH, s.X, s.Wg, s.Wu, s.G, s.U, plan, weights=s.w, dX=dX.t,
                                      dWg=dW[1:E + 1], dWu=dV[1:E + 1], dweights=dw.t)
    for b in (H, Y, dH, dX, dw):
        b.check()
    for t in (dW, dV, dD):
        assert bool((t[0] == 7).all()) and bool((t[-1] == 7).all())
    # the inputs are as they were, and so are the results of the right plan
    near(lm.llmint8_experts_matmul(s.H, s.Wd, s.plan),
         eo.matmul(s.H.double(), s.Wd.double(), s.p, None, F16, s.rounded))


def test_workspaces_of_their_size(lm):
    """A call stays within the workspace that the query names, and refuses a smaller one."""
    say("workspaces")
    for M, K, N, E, k in ((1, 4096, 136, 8, 2), (300, 264, 520, 20, 3), (2000, 264, 136, 4, 2)):
        s = Experts(lm, M, K, N, E, k, 0.0, BF16)
        calls = dict(
            gated=lambda ws: lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, s.plan, weights=s.w,
                                                      workspace=ws),
            matmul=lambda ws: lm.llmint8_experts_matmul(s.H, s.Wd, s.plan, workspace=ws),
            matmul_backward=lambda ws: lm.llmint8_experts_matmul_backward(
                s.dY, s.H, s.Wd, s.plan, workspace=ws),
            gated_backward=lambda ws: lm.llmint8_experts_gated_backward(
                s.dH, s.X, s.Wg, s.Wu, s.G, s.U, s.plan, weights=s.w, workspace=ws))
        for name, call in calls.items():
            need = getattr(lm, f"llmint8_experts_{name}_workspace_size")(M, K, N, E, k)
            held = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
            got, want = call(held[4096:4096 + need] if need else None), call(None)
            torch.cuda.synchronize()
            assert bool((held[:4096] == 0xA5).all()) and bool((held[4096 + need:] == 0xA5).all())
            for a, b in zip(got if isinstance(got, tuple) else (got,),
                            want if isinstance(want, tuple) else (want,)):
                assert torch.equal(a, b), name
            if need:
                with pytest.raises((ValueError, lm.Llmint8Error)):
                    call(held[4096:4096 + need - 16])


@pytest.mark.parametrize("M,K,N,E,k", [(1, 264, 136, 6, 4), (300, 136, 264, 30, 3),
                                       (3000, 136, 264, 5, 3)])
def test_not_finite(lm, M, K, N, E, k):
    """A token with a NaN, an expert with one: no other row shows it, forward or backward."""
    say("not finite", M, K, N, E, k)
    s = Experts(lm, M, K, N, E, k, 0.0, F16)
    i, e = M // 2, int(s.ids[0, 0])
    clean = lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, s.plan, weights=s.w)
    for bad in (math.nan, math.inf):
        X = s.X.clone()
        X[i, 5] = bad
        rows = s.plan.places[i].long()
        keep = torch.ones(M * k, dtype=torch.bool, device="cuda")
        keep[rows] = False
        h = lm.llmint8_experts_gated(X, s.Wg, s.Wu, s.plan, weights=s.w)
        assert torch.equal(h[keep], clean[keep])
        assert not bool(torch.isfinite(h[rows]).all(1).any())
        Wg = s.Wg.clone()
        Wg[e, 3, 7] = bad
        mine = slice(int(s.p[0][e]), int(s.p[0][e + 1]))
        h = lm.llmint8_experts_gated(s.X, Wg, s.Wu, s.plan, weights=s.w)
        same = torch.ones(M * k, dtype=torch.bool, device="cuda")
        same[mine] = False
        assert torch.equal(h[same], clean[same])
        # a token's gradient reaches its experts' weights and no others'
        dY = s.dY.clone()
        dY[i, 2] = bad
        a = lm.llmint8_experts_matmul_backward(dY, s.H, s.Wd, s.plan)
        b = lm.llmint8_experts_matmul_backward(s.dY, s.H, s.Wd, s.plan)
        assert torch.equal(a[0][keep], b[0][keep])
        others = [x for x in range(E) if x not in s.ids[i].tolist()]
        assert torch.equal(a[1][others], b[1][others])


@pytest.mark.parametrize("name", fo.ACTS)
def test_every_activation(lm, name):
    """Few rows, in one part and in several, and tiles; forward and backward."""
    say("activation", name)
    for M, K, N, E, k in ((1, 4096, 136, 3, 2), (60, 264, 136, 6, 2), (3000, 136, 264, 5, 2)):
        s = Experts(lm, M, K, N, E, k, 0.0, BF16)
        h = lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, s.plan, weights=s.w, activation=name)
        near(h, eo.gated(s.X.double(), s.Wg.double(), s.Wu.double(), s.p, s.w, name, BF16)["H"])
        got = lm.llmint8_experts_gated_backward(s.dH, s.X, s.Wg, s.Wu, s.G, s.U, s.plan,
                                                weights=s.w, activation=name)
        want = eo.gated_backward(s.dH.double(), s.X.double(), s.Wg.double(), s.Wu.double(),
                                 s.G.double(), s.U.double(), s.p, s.w, name, BF16)
        for t, n in zip(got, ("dX", "dWg", "dWu", "dw")):
            near(t, want[n])
    with pytest.raises(ValueError):
        lm.llmint8_experts_gated(s.X, s.Wg, s.Wu, s.plan, activation="swish")


def test_broadcast_weights(lm):
    """One expert's weights for all (a stride of 0), and no such output."""
    say("broadcast")
    for M, K, N, E, k in ((5, 264, 136, 6, 2), (900, 136, 264, 3, 2)):
        s = Experts(lm, M, K, N, E, k, 0.0, BF16)
        Wg, Wu, Wd = (t[:1].expand(E, -1, -1) for t in (s.Wg, s.Wu, s.Wd))
        a = lm.llmint8_experts_gated(s.X, Wg, Wu, s.plan)
        assert torch.equal(a, lm.llmint8_experts_gated(s.X, Wg.contiguous(), Wu.contiguous(), s.plan))
        assert torch.equal(lm.llmint8_experts_matmul(s.H, Wd, s.plan),
                           lm.llmint8_experts_matmul(s.H, Wd.contiguous(), s.plan))
        out = torch.zeros_like(s.Wd)[:1].expand(E, -1, -1)
        with pytest.raises(lm.Llmint8Error):
            lm.llmint8_experts_matmul_backward(s.dY, s.H, s.Wd, s.plan, dWd=out)


# ---- past 2 GiB and 2^32 elements -------------------------------------------------------

@pytest.mark.parametrize("M,K,N,E", [(131077, 8192, 16, 3), (66000, 16384, 8, 1024)])
def test_tokens_past_2_gib(lm, M, K, N, E):
    """X and dX of more than 2^31 bytes; every value at sampled rows, the gradients of the
    weights of sampled experts whole."""
    say("past 2 GiB", M, K, N, E)
    torch.cuda.empty_cache()
    g = gen(1)
    X = torch.randn((M, K), generator=g, device="cuda", dtype=BF16)
    assert X.numel() * 2 >= 2 ** 31
    Wg, Wu, Wd = (rand(g, E * a, b, BF16, 0.02).view(E, a, b) for a, b in ((K, N), (K, N), (N, K)))
    ids = torch.randint(0, E, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    plan = lm.llmint8_expert_plan(ids, E)
    w = torch.rand((M, 1), generator=g, device="cuda")
    H, G, U = lm.llmint8_experts_gated(X, Wg, Wu, plan, weights=w, save="full")
    Y = lm.llmint8_experts_matmul(H, Wd, plan, residual=X)
    dH = rand(g, M, N, BF16)
    dX, dWg, _, dw = lm.llmint8_experts_gated_backward(dH, X, Wg, Wu, G, U, plan, weights=w)
    at = torch.cat([torch.tensor([0, 1, M - 2, M - 1]), torch.randint(0, M, (60,))]).cuda()
    at = at.unique()
    n = at.numel()
    sub = ids[at]
    p = eo.plan(sub, E)
    mine = plan.places[at, 0].long()[p[1].long()]  # the rows of the small plan's rows
    want = eo.gated(X[at].double(), Wg.double(), Wu.double(), p, w[at], "silu", BF16)
    for t, name in ((H, "H"), (G, "G"), (U, "U")):
        near(t[mine], want[name])
    near(Y[at], eo.matmul(H[mine].double(), Wd.double(), p, X[at].double(), BF16, True))
    back = eo.gated_backward(dH[mine].double(), X[at].double(), Wg.double(), Wu.double(),
                             G[mine].double(), U[mine].double(), p, w[at], "silu", BF16)
    near(dX[at], back["dX"]), near(dw[at], back["dw"])
    for e in (0, E - 1):
        tok = (ids[:, 0] == e).nonzero()[:, 0]
        r = plan.places[tok, 0].long()
        one = eo.plan(torch.zeros((tok.numel(), 1), dtype=torch.int32, device="cuda"), 1)
        small = eo.gated_backward(dH[r].double(), X[tok].double(), Wg[e:e + 1].double(),
                                  Wu[e:e + 1].double(), G[r].double(), U[r].double(), one, w[tok],
                                  "silu", BF16)
        near(dWg[e:e + 1], small["dWg"])
    assert n > 4
    torch.cuda.empty_cache()


def test_strides_past_2_32(lm):
    """Rows and experts whose distances add up to more than 2^32 bytes; X of that span is refused
    unless its rows follow one another."""
    say("strides past 2^32")
    torch.cuda.empty_cache()
    M, K, N, E, k = 2500, 136, 72, 3, 2
    s = Experts(lm, M, K, N, E, k, 0.0, F16)
    far = lambda t: torch.empty(  # noqa: E731
        (E * 2 ** 31,), dtype=F16, device="cuda").as_strided(t.shape, (2 ** 31, t.shape[2] + 8, 1))
    wide = lambda t, ld=2 ** 20: torch.empty(  # noqa: E731
        (t.shape[0] * ld,), dtype=t.dtype, device="cuda").as_strided(t.shape, (ld, 1))
    Wg, H = far(s.Wg).copy_(s.Wg), wide(s.H)
    Wu = far(s.Wu).copy_(s.Wu)
    lm.llmint8_experts_gated(s.X, Wg, Wu, s.plan, weights=s.w, H=H)
    near(H, eo.gated(s.X.double(), s.Wg.double(), s.Wu.double(), s.p, s.w, "silu", F16)["H"])
    H.copy_(s.H)
    Y, dWd = wide(s.R), far(s.Wd)
    lm.llmint8_experts_matmul(H, s.Wd, s.plan, Y=Y)
    near(Y, eo.matmul(s.H.double(), s.Wd.double(), s.p, None, F16, s.rounded))
    dH = wide(s.dH)
    dY = wide(s.dY).copy_(s.dY)
    lm.llmint8_experts_matmul_backward(dY, H, s.Wd, s.plan, dH=dH, dWd=dWd)
    want = eo.matmul_backward(s.dY.double(), s.H.double(), s.Wd.double(), s.p, F16)
    near(dH, want["dH"]), near(dWd, want["dWd"])
    X = wide(s.X).copy_(s.X)
    with pytest.raises(lm.Llmint8Error) as e:
        lm.llmint8_experts_gated(X, s.Wg, s.Wu, s.plan)
    assert e.value.status == lm.LLMINT8_ERR_UNSUPPORTED
    # the router's logits, and the backward pass's X, may span more
    dX, dWg, _, _ = lm.llmint8_experts_gated_backward(s.dH, X, s.Wg, s.Wu, s.G, s.U, s.plan,
                                                      weights=s.w)
    want = eo.gated_backward(s.dH.double(), s.X.double(), s.Wg.double(), s.Wu.double(),
                             s.G.double(), s.U.double(), s.p, s.w, "silu", F16)
    near(dX, want["dX"]), near(dWg, want["dWg"])
    x = torch.randn((M, 64), generator=gen(4), device="cuda")
    logits = wide(x).copy_(x)
    ids, w = lm.llmint8_route(logits, 6)
    assert torch.equal(ids, eo.choose(x, 6))
    near(w, eo.mix(x, ids, "softmax", False))
    near(lm.llmint8_route_backward(w, logits, ids, dlogits=wide(x)),
         eo.route_backward(w, x, ids, "softmax", False, 1.0))
    del Wg, Wu, H, Y, dWd, dH, dY, X, logits
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [1, 130])
def test_block_scaled_weights_past_2_31(lm, M):
    say("fp8 past 2^31", M)
    torch.cuda.empty_cache()
    K, N = 131072, 16400
    g = gen(M)
    wq = torch.randint(0, 126, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    wq[:, ::2] += 128
    sw = torch.randint(110, 120, (-(-N // 128), K // 128), generator=g, device="cuda").to(torch.uint8)
    big = torch.empty((M * 2 ** 20,), dtype=BF16, device="cuda")
    x = big.as_strided((M, K), (2 ** 20, 1)).copy_(rand(g, M, K, BF16))
    y = lm.llmint8_linear_blockwise_fp8(x, wq, sw)
    for n0 in (0, 8192, N - 144):  # whole blocks of columns
        n1 = min(n0 + 144, N)
        b0 = n0 // 128
        codes = wq[b0 * 128:n1].contiguous()
        want, tol = bo.linear(x, codes, sw[b0:-(-n1 // 128)], None, BF16)
        near(y[:, n0:n1], (want[:, n0 - b0 * 128:], tol[:, n0 - b0 * 128:]))
    torch.cuda.empty_cache()


def test_training_example():
    """The example runs, and its gradients are those of 64 bits with the choice held."""
    say("training example")
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_routed_feed_forward.py")
    spec = importlib.util.spec_from_file_location("train_routed_feed_forward", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, W, bias = ex.train(steps=3, tokens=100, width=64, hidden=40, experts=8, k=2, dtype=F16)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
    g = gen(9)
    X, D = rand(g, 60, 64, F16), rand(g, 60, 64, F16, 0.1)
    Y, saved = ex.forward(X, W, 2, bias, keep=True)
    assert torch.equal(Y, ex.forward(X, W, 2, bias)[0])
    grads, dX = ex.backward(D, W, saved)
    ids = saved[2].long()
    x, *w = [t.detach().double().cpu().requires_grad_() for t in (X, *W)]
    s = torch.sigmoid(torch.gather(x @ w[0], 1, ids.cpu()))
    s = s / s.sum(1, keepdim=True)
    y = x
    for e in range(8):
        h = fo.act("silu", x @ w[1][e]) * (x @ w[2][e])
        y = y + (s * (ids.cpu() == e)).sum(1, keepdim=True) * (h @ w[3][e])
    (y * D.double().cpu()).sum().backward()
    # independent roundings of 2^-11, a dozen at most one after the other (logits, G, U, H, dH,
    # dG, dU, dlogits and the results), of which the logits' is multiplied by what w (1 - s) and
    # the gradients' cancellation over the chosen make of it: a hundredth of the norm
    for name, got, want in zip(("dX", "dWr", "dWg", "dWu", "dWd"), (dX, *grads), (x, *w)):
        got, want = got.double().cpu(), want.grad
        assert float((got - want).norm()) <= 0.01 * float(want.norm()), name
