"""The block-scaled FP8 product at the ends of the scales' range: a row's scale and a column block's
far apart, whose product is an ordinary number. The entries are 0 or a power of two, so the sums are
whole multiples of it and exact."""
import pytest
import torch

import fp8_block_oracle as bo
from test_ffn_gpu import BF16, gen, lm, say  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", [(1, 1040, 520), (40, 528, 264), (200, 1040, 264), (600, 272, 2056),
                                   (2100, 528, 5128)])
@pytest.mark.parametrize("e", [-127, -126, -119, -118, -90, 90, 120, 126, 127])
def test_scales_far_apart(lm, M, K, N, e):
    say("scales far apart", M, K, N, e)
    g = gen(M + K)
    x = torch.randint(-1, 2, (M, K), generator=g, device="cuda").double() * 2.0 ** e
    x = x.to(BF16)
    codes = torch.randint(0, 3, (N, K), generator=g, device="cuda")
    wq = torch.tensor([0, 0x38, 0xb8], dtype=torch.uint8, device="cuda")[codes]  # 0, 1, -1
    byte = 127 - e
    nb, kb = -(-N // 128), -(-K // 128)
    sw = torch.full((nb, kb), byte, dtype=torch.uint8, device="cuda")
    y = lm.llmint8_linear_blockwise_fp8(x, wq, sw)
    want = x.double() @ bo.values(wq, bo.spread_weights(sw, N, K)).t()
    assert float(want.abs().max()) < 2 * K
    assert torch.equal(y, want.to(BF16))
