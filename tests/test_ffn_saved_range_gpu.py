"""8-bit checkpoints whose entries do not fit the 16-bit type they are expanded to:
pre-activations taken from fp32 sums, and bf16 activations expanded to fp16. Expanding
rounds the value code * 2^e once (to infinity past the type's end); the backward pass of
the gated block takes G and U as they are."""
import pytest
import torch

import ffn_oracle as fo
import test_ffn_gpu as base

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def lm():
    import bit_quantized_matmul_col_amd as lm
    lm.lib()
    return lm


# sums of about 2^-26, below fp16's subnormal step, and of 10^5, past its end
@pytest.mark.parametrize("size", [2.0 ** -13, 100.0])
@pytest.mark.parametrize("M", [5, 300])
def test_gated_sums_outside_fp16(lm, M, size):
    base.say("saved range", M, size)
    g = base.gen(7)
    K, N = 16, 72
    X, Wg, Wu = (base.rand(g, a, b, F16, size).clamp(-250, 250) for a, b in ((M, K), (K, N), (K, N)))
    _, G, U = lm.llmint8_gated(X, Wg, Wu, activation="relu", save="8bit")
    _, (want_g, err_g), (want_u, err_u) = fo.gated(X.double(), Wg.double(), Wu.double(), "relu", F16)
    values = []
    for c, want, err in ((G, want_g, err_g), (U, want_u, err_u)):
        v = fo.unpack(c.codes, c.scales)
        step = fo.pow2(c.scales.long() - 127).repeat_interleave(32, dim=1)[:, :N]
        base.near(v, (want, step + err))
        half = v.float().to(F16)
        assert not torch.equal(half.double(), v), "the test's values fit fp16 after all"
        back = lm.llmint8_checkpoint_unpack(c, F16)
        assert torch.equal(back, half)
        assert bool(back.isinf().any()) == (size > 1)
        assert torch.equal(lm.llmint8_checkpoint_unpack(c, BF16).double(), v), "exact in bf16"
        values.append(v)
    dH = base.rand(g, M, N, F16, 2.0 ** -12 if size > 1 else 2.0 ** 12)
    W2 = base.rand(g, K, N, F16, 0.05)
    Xb = base.rand(g, M, K, F16)
    got = lm.llmint8_gated_backward(dH, Xb, W2, W2, G, U, activation="relu")
    want = fo.gated_backward(dH.double(), Xb.double(), W2.double(), W2.double(), *values, "relu", F16)
    for a, w in zip(got, want):
        assert bool(a.isfinite().all())
        base.near(a, w)


def test_bf16_checkpoint_expanded_to_fp16(lm):
    base.say("bf16 to fp16")
    g = base.gen(8)
    X = base.rand(g, 6, 96, BF16)
    X[0] *= 2.0 ** -20
    X[1] *= 2.0 ** -40
    X[2] *= 2.0 ** 15
    X[3] *= 2.0 ** 100
    c = lm.llmint8_checkpoint_pack(X)
    v = fo.unpack(c.codes, c.scales)
    assert torch.equal(lm.llmint8_checkpoint_unpack(c, BF16).double(), v)
    assert torch.equal(lm.llmint8_checkpoint_unpack(c, F16), v.float().to(F16))
