"""Block-scaled FP8 on the GPU: codes and scales bit for bit, the product within the bound
of tests/fp8_block_oracle.py, on every kernel path."""
import math

import pytest
import torch

import ffn_oracle as fo
import fp8_block_oracle as bo
from test_ffn_gpu import BF16, F16, Band, gen, lm, near, rand, say, strided  # noqa: F401

pytestmark = pytest.mark.gpu


def wide(g, M, K, dtype):
    """Entries over many binades, block by block, and some blocks of zeros."""
    x = torch.randn((M, K), generator=g, device="cuda")
    lo, hi = (-20, 10) if dtype is F16 else (-60, 60)
    e = torch.randint(lo, hi, (M, -(-K // 32)), generator=g, device="cuda").float()
    x = x * torch.exp2(e).repeat_interleave(32, 1)[:, :K]
    x[torch.rand((M, K), generator=g, device="cuda") < 0.05] = 0
    if K > 128:
        x[M // 2, :128] = 0
    return x.clamp(min=-60000 if dtype is F16 else -1e38, max=60000 if dtype is F16 else 1e38).to(dtype)


SIZES = [(1, 16, 8), (3, 48, 24), (128, 128, 128), (37, 528, 264), (130, 1040, 520), (257, 144, 1000)]


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_codes(lm, M, K, N, dtype):
    say("fp8 codes", M, K, N, dtype)
    g = gen(M + K + N)
    for make in (rand, wide):
        x, w = make(g, M, K, dtype), make(g, K, N, dtype)
        q, s = lm.llmint8_quantize_rowblock_fp8(strided(x))
        want, byte = bo.rows(x)
        assert torch.equal(s.long(), byte) and torch.equal(q.long(), want)
        q, s = lm.llmint8_quantize_blockwise_fp8(strided(w))
        want, byte = bo.weights(w)
        assert torch.equal(s.long(), byte) and torch.equal(q.long(), want)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_every_value_and_the_edges_of_the_scale(lm, dtype):
    """Blocks with every finite 16-bit value as the largest, then as any entry."""
    say("fp8 every value", dtype)
    bits = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    v = bits[torch.isfinite(bits)]
    x = torch.zeros((v.numel(), 16), dtype=dtype, device="cuda")
    x[:, 3] = v
    x[:, 7] = v / 3
    q, s = lm.llmint8_quantize_rowblock_fp8(x)
    want, byte = bo.rows(x)
    assert torch.equal(s.long(), byte) and torch.equal(q.long(), want)
    # 448 and 1 in the block: every value up to 448 meets the scale 1
    small = v[v.abs() <= 448]
    x = torch.zeros((small.numel(), 16), dtype=dtype, device="cuda")
    x[:, 0], x[:, 1] = 448, small
    q, s = lm.llmint8_quantize_rowblock_fp8(x)
    assert int(s.min()) == int(s.max()) == 127
    assert torch.equal(q.long(), bo.rows(x)[0])


# M, K, N: few rows in one launch and coded before, with 16, 32 and 64 columns a block; tiles of 128
# with rings of two and four stages, whole and split; tiles of 256; odd sizes on every side
PRODUCTS = [(1, 16, 8), (1, 4096, 4096), (1, 1040, 28680), (5, 11008, 264), (16, 528, 8200),
            (17, 272, 136), (24, 2064, 16392), (33, 1040, 520), (64, 4096, 1032), (100, 144, 8200),
            (129, 1040, 264), (200, 8208, 136), (300, 528, 4104), (513, 2064, 1032),
            (1000, 272, 1096), (1500, 1040, 4104), (2049, 144, 4104), (2100, 4112, 5128),
            (700, 11008, 520), (4097, 32, 264), (128, 12304, 3336), (140, 16, 14344)]


@pytest.mark.parametrize("M,K,N", PRODUCTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_linear(lm, M, K, N, dtype):
    say("fp8 linear", M, K, N, dtype)
    g = gen(M + 2 * K + 3 * N)
    x, w = rand(g, M, K, dtype), rand(g, K, N, dtype, 0.05)
    x[:, K // 3] *= 40
    bias = rand(g, 1, N, dtype)[0]
    wq, sw = lm.llmint8_quantize_blockwise_fp8(w)
    Y = Band(M, N, dtype)
    lm.llmint8_linear_blockwise_fp8(strided(x), wq, sw, bias=bias, Y=Y.t)
    Y.check()
    near(Y.t, bo.linear(x, wq, sw, bias, dtype))
    a = lm.llmint8_linear_blockwise_fp8(x, wq, sw)
    assert torch.equal(a, lm.llmint8_linear_blockwise_fp8(x, wq, strided8(sw)))
    near(a, bo.linear(x, wq, sw, None, dtype))


def strided8(s):
    big = torch.full((s.shape[0], s.shape[1] + 3), 255, dtype=torch.uint8, device=s.device)
    big[:, :s.shape[1]] = s
    return big[:, :s.shape[1]]


@pytest.mark.parametrize("M,K,N", [(1, 1040, 520), (40, 528, 264), (200, 1040, 264), (600, 272, 2056),
                                   (2100, 528, 5128)])
def test_units_are_exact(lm, M, K, N):
    """Entries of 0 and +-1 at scales over many binades: the sums are whole numbers that an
    MFMA holds, so each block's scale is seen exactly."""
    say("fp8 units", M, K, N)
    g = gen(M + K)
    kb, nb = -(-K // 128), -(-N // 128)
    x = torch.randint(-1, 2, (M, K), generator=g, device="cuda").to(BF16)
    # one power of two a row or column block, so that sums of a row stay exact
    ex = torch.randint(-30, 30, (M, 1), generator=g, device="cuda").float()
    x = (x.float() * torch.exp2(ex)).to(BF16)
    codes = torch.randint(0, 3, (N, K), generator=g, device="cuda")
    wq = torch.tensor([0, 0x38, 0xb8], dtype=torch.uint8, device="cuda")[codes]
    sw = torch.randint(100, 150, (nb, 1), generator=g, device="cuda").expand(nb, kb)
    sw = sw.to(torch.uint8).contiguous()
    y = lm.llmint8_linear_blockwise_fp8(x, wq, sw)
    wv = bo.values(wq, bo.spread_weights(sw, N, K))
    assert torch.equal(y, (x.double() @ wv.t()).to(BF16))


@pytest.mark.parametrize("M", [1, 40, 200, 2100])
def test_not_finite(lm, M):
    """An infinity or a NaN makes its block NaN, in its row (column) alone; other rows and the gap
    between rows do not show."""
    say("fp8 not finite", M)
    K, N = 1040, 5128
    g = gen(M)
    x, w = rand(g, M, K, F16), rand(g, K, N, F16, 0.05)
    w[5, 7] = math.inf
    wq, sw = lm.llmint8_quantize_blockwise_fp8(w)
    assert int(sw[0, 0]) == 255 and bool((wq[:128, :128] == 0x7f).all())
    x[M - 1, 1030] = math.nan
    y = lm.llmint8_linear_blockwise_fp8(strided(x), wq, sw)
    nan = torch.isnan(y)
    assert bool(nan[:, :128].all()) and bool(nan[M - 1].all())
    assert not bool(nan[:M - 1, 128:].any())
    if M > 1:
        clean = lm.llmint8_quantize_blockwise_fp8(torch.where(torch.isfinite(w), w, 0 * w))
        ref, tol = bo.linear(x[:M - 1], *clean, None, F16)
        near(y[:M - 1, 128:], (ref[:, 128:], tol[:, 128:]))
