"""A rank that holds a part of the experts: ids of the others are none of its own, so most pairs
have no row. Where it holds fewer experts than a token chooses, it names k of them, the ones
past its own without rows and at a weight stride of 0. And what a bias that is not finite
does to the choice."""
import math

import pytest
import torch

import experts_oracle as eo
from test_experts_gpu import rows_only
from test_ffn_gpu import BF16, F16, gen, lm, near, rand, say  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N,E,k,held", [(1, 264, 136, 8, 2, 1), (40, 136, 520, 64, 6, 8),
                                            (700, 264, 136, 8, 4, 1), (4100, 136, 264, 8, 3, 2),
                                            (3000, 520, 264, 128, 8, 16)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_part_of_the_experts(lm, M, K, N, E, k, held, dtype):
    say("part of the experts", M, K, N, E, k, held, dtype)
    g = gen(M + E)
    all_ids = torch.rand((M, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    named = max(held, k)
    X, dY = rand(g, M, K, dtype), rand(g, M, K, dtype, 0.5)
    w = torch.rand((M, k), generator=g, device="cuda")
    some = False
    for first in (0, E - held):
        ids = all_ids - first
        ids[(ids < 0) | (ids >= held)] = -1
        plan, p = lm.llmint8_expert_plan(ids, named), eo.plan(ids, named)
        for a, b in zip(plan, p):
            assert torch.equal(a, b)
        last = int(p[0][-1])
        some |= last > 0
        own = [rand(g, held * a, b, dtype, 0.1).view(held, a, b) for a, b in ((K, N), (K, N), (N, K))]
        Wg, Wu, Wd = (t.expand(named, -1, -1) if held == 1 else
                      t if named == held else torch.cat([t, t[:1].expand(named - held, -1, -1)])
                      for t in own)
        H, G, U = lm.llmint8_experts_gated(X, Wg, Wu, plan, weights=w, save="full")
        want = eo.gated(X.double(), Wg.double(), Wu.double(), p, w, "silu", dtype)
        for n, t in (("H", H), ("G", G), ("U", U)):
            rows_only(t, want[n], last)
        for t in (H, G, U):
            t[last:] = 0  # for the definitions below; no call reads these rows
        near(lm.llmint8_experts_matmul(H, Wd, plan),
             eo.matmul(H.double(), Wd.double(), p, None, dtype, False))
        dH, dWd = lm.llmint8_experts_matmul_backward(dY, H, Wd, plan)
        want = eo.matmul_backward(dY.double(), H.double(), Wd.double(), p, dtype)
        rows_only(dH, want["dH"], last)
        near(dWd, want["dWd"])
        dH[last:] = 0
        out = lm.llmint8_experts_gated_backward(dH, X, Wg, Wu, G, U, plan, weights=w)
        want = eo.gated_backward(dH.double(), X.double(), Wg.double(), Wu.double(), G.double(),
                                 U.double(), p, w, "silu", dtype)
        for n, t in zip(("dX", "dWg", "dWu", "dw"), out):
            near(t, want[n])
        for t in (dWd, out[1], out[2]):
            assert not bool(t[held:].any())
    assert some or M == 1


@pytest.mark.parametrize("groups,top,best", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_a_bias_that_is_not_finite(lm, groups, top, best, scores):
    """-infinity or NaN: never chosen, and nothing to a group's value; the scores are as without."""
    say("bias not finite", groups, best, scores)
    g = gen(groups + best)
    M, E, k = 70, 64, 6
    x = torch.randn((M, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
    bias[8:16] = -math.inf  # a whole group
    bias[[0, 5, 33]] = -math.inf
    want = eo.choose(x, k, scores, bias, groups, top, best)
    assert not bool(((want >= 8) & (want < 16)).any())
    for bad in (-math.inf, math.nan):
        b = torch.where(torch.isfinite(bias), bias, torch.full_like(bias, bad))
        ids, w = lm.llmint8_route(x, k, scores=scores, bias=b, groups=groups, top_groups=top,
                                  group_best=best)
        assert torch.equal(ids, want)
        near(w, eo.mix(x, ids, scores, False))
    none = torch.full((E,), -math.inf, device="cuda")
    ids, w = lm.llmint8_route(x, k, scores=scores, bias=none, groups=groups, top_groups=top,
                              group_best=best)
    assert bool((ids == -1).all()) and not bool(w.any())
