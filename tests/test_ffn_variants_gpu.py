"""The kernel variants of the 16-bit feed-forward operators that the shapes of
test_ffn_gpu.py do not take, held to the same definitions and bounds by the same
checks. test_ffn_plan_cpu.py asks the plan which variants the two files reach."""
import pytest
import torch

import test_ffn_gpu as base

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16

# M, K, N: few rows in groups of 32 with blocks of 128 columns, whole and split; 128-tiles
# in a ring of four stages and 256-tiles, split
FORWARD = [(17, 24, 16456), (533, 1296, 24), (18, 4904, 2704), (17, 9176, 3784),
           (134, 3272, 16496), (31, 5480, 12040), (704, 7664, 4056), (2048, 11008, 4096)]

# Both products of a backward pass in one launch: 128- and 256-tiles, rings of two and four
# stages, either product split, both and neither, either of them first; each product alone
BACKWARD = [(1871, 3224, 24), (1, 24, 1160), (1111, 24, 280), (338, 24, 1328), (403, 19104, 24),
            (1953, 24, 1608), (1565, 24, 2504), (3011, 24, 5504), (1, 11160, 1416),
            (2066, 24, 7864), (1015, 1296, 136), (213, 1072, 1552), (965, 1680, 272),
            (193, 20120, 136), (3150, 1928, 400), (418, 14440, 400), (389, 15528, 408),
            (8085, 136, 7016), (3481, 1880, 400), (751, 1272, 2984), (5284, 144, 10936),
            (496, 1704, 4992), (2248, 3016, 648), (2772, 2488, 664), (739, 2528, 2952),
            (7672, 136, 8000), (2048, 4096, 4096)]


@pytest.fixture(scope="module")
def lm():
    import bit_quantized_matmul_col_amd as lm
    lm.lib()
    return lm


@pytest.mark.parametrize("M,K,N", FORWARD)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_matmul(lm, M, K, N, dtype):
    base.test_matmul(lm, M, K, N, dtype)


@pytest.mark.parametrize("M,K,N", FORWARD)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gated(lm, M, K, N, dtype):
    base.test_gated(lm, M, K, N, dtype)


# the bias gradient's end among the tiles gives the bits of the kernel that does it alone
@pytest.mark.parametrize("M,K,N", BACKWARD)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_matmul_backward(lm, M, K, N, dtype):
    base.test_matmul_backward(lm, M, K, N, dtype, "full")


@pytest.mark.parametrize("M,K,N", BACKWARD)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gated_backward(lm, M, K, N, dtype):
    base.test_gated_backward(lm, M, K, N, dtype, "full")


def test_more_rows_than_the_grid_has(lm):
    """70001 rows of one row a block: the row-streaming passes stride over a grid of 65535."""
    M, K, N = 70001, 24, 2056
    base.test_checkpoint(lm, M, N, BF16)
    base.test_matmul(lm, M, K, N, BF16)
    base.test_gated(lm, M, K, N, F16)
    base.test_matmul_backward(lm, M, K, N, F16, "8bit")
    base.test_gated_backward(lm, M, K, N, BF16, "8bit")
