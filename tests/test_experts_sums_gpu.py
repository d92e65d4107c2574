"""The sum over a token's experts rounds once, whichever kernel computes the rows. The operands are
small whole numbers, so that every row and every sum is exact in fp32 and the result is the
exact sum's one rounding; a token's first two rows are large (beyond fp16's range) and
cancel, so a row that went through 16 bits would show as an infinity, a NaN or a wrong entry."""
import pytest
import torch

from test_ffn_gpu import BF16, F16, Band, gen, lm, say  # noqa: F401

pytestmark = pytest.mark.gpu

# M, columns, reduction, E, k: few rows of 16, 32 and 64 a group, in one part and in several; tiles
# of 128 and of 256 rows, with a last one that is not full; more choices than two
SHAPES = [(1, 264, 136, 8, 2), (2, 136, 4096, 6, 2), (60, 520, 264, 6, 3), (333, 520, 1040, 11, 3),
          (700, 136, 264, 4, 2), (513, 264, 136, 2, 2), (3000, 264, 136, 5, 4),
          (4097, 520, 264, 16, 2)]


def whole(g, low, high, *shape):
    return torch.randint(low, high, shape, generator=g, device="cuda").double()


class Cancelling:
    """Rows v [M, k, n] of which a token's first is 100 .. 249 and its second minus that, but for -1,
    0 or 1, the others -2 .. 2; every seventh token has no expert. All whole numbers."""

    def __init__(self, lm, M, n, E, k, seed):
        g = gen(seed + M + n)
        ids = torch.rand((M, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
        ids[3::7] = -1
        self.plan = lm.llmint8_expert_plan(ids.contiguous(), E)
        self.v = whole(g, -2, 3, M, k, n)
        self.v[:, 0] = whole(g, 100, 250, M, n)
        self.v[:, 1] = whole(g, -1, 2, M, n) - self.v[:, 0]
        self.v[3::7] = 0
        self.g = g

    def rows(self, dtype, scale=1):
        """scale v in the plan's order, NaN behind the last row."""
        at = self.plan.places.reshape(-1).long()
        M, k, n = self.v.shape
        out = torch.full((M * k, n), float("nan"), dtype=dtype, device="cuda")
        v = (scale * self.v).to(dtype)
        assert torch.equal(v.double(), scale * self.v)
        out[at[at >= 0]] = v.view(M * k, n)[at >= 0]
        return out


@pytest.mark.parametrize("M,K,N,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_second_product_of_rows_that_cancel(lm, M, K, N, E, k, dtype):
    say("rows that cancel", M, K, N, E, k, dtype)
    s = Cancelling(lm, M, N, E, k, 0)
    B, R = whole(s.g, 1, 9, N, K), whole(s.g, -200, 201, M, K)
    row = s.v[:, 0] @ B
    assert float(row.max()) > 65504 and 2 * float(row.max()) < 2 ** 24
    Wd = B.to(dtype).expand(E, -1, -1).contiguous()
    want = s.v.sum(1) @ B
    Y = Band(M, K, dtype)
    lm.llmint8_experts_matmul(s.rows(dtype), Wd, s.plan, residual=R.to(dtype), Y=Y.t)
    Y.check()
    assert torch.equal(Y.t, (want + R).to(dtype))
    assert torch.equal(lm.llmint8_experts_matmul(s.rows(dtype), Wd, s.plan), want.to(dtype))


@pytest.mark.parametrize("M,K,N,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradient_of_rows_that_cancel(lm, M, K, N, E, k, dtype):
    """dX, likewise: without an activation, with G = 1, U = 2 and weights of a half, dG = dH and
    dU = dH / 2 are whole numbers of 16 bits, so that nothing rounds but the sum."""
    say("gradient rows that cancel", M, K, N, E, k, dtype)
    s = Cancelling(lm, M, N, E, k, 1)
    Bg, Bu = whole(s.g, 1, 5, K, N), whole(s.g, 1, 9, K, N)
    both = (2 * Bg + Bu).t()
    row = s.v[:, 0] @ both
    assert float(row.max()) > 65504 and 2 * float(row.max()) < 2 ** 24
    Wg, Wu = (t.to(dtype).expand(E, -1, -1).contiguous() for t in (Bg, Bu))
    one = torch.ones((M * k, N), dtype=dtype, device="cuda")
    half = torch.full((M, k), 0.5, device="cuda")
    dX = Band(M, K, dtype)
    lm.llmint8_experts_gated_backward(s.rows(dtype, 2), None, Wg, Wu, one, 2 * one, s.plan,
                                      weights=half, activation="none", dX=dX.t, need_dW=False)
    dX.check()
    assert torch.equal(dX.t, (s.v.sum(1) @ both).to(dtype))
