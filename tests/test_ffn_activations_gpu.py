"""The smooth activations and their derivatives at every fp16 and bf16 argument of their
range, in relative terms: the lower tails, where 1 + erf and 1 + tanh cancel, are as
accurate as the rest.

act(z) = z p(z), p the normal distribution (gelu) or the logistic function of w(z) (silu,
w = z; gelu_tanh, w = 2 sqrt(2 / pi) (z + 0.044715 z^3)). The bound, relative: p is held
to 2^-19 (a handful of fp32 roundings and 1 ulp each for the hardware exponential and
reciprocal) and, through the exponent (z^2 / 2, or w), whose at most seven roundings of
2^-24 change p by as many of the exponent, to 2^-21 of the exponent; then one rounding to
16 bits. The derivative p + z p' has that of its two terms, and where z is positive that
of 1 - p = 2^-23 times the rest of the second."""
import math

import pytest
import torch

import ffn_oracle as fo

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
TANH = 2 * math.sqrt(2 / math.pi)
# up to where the exponential of the lower tail is a normal fp32 number
TOP = {"gelu": 12.75, "gelu_tanh": 9.75, "silu": 80.0}


@pytest.fixture(scope="module")
def lm():
    import bit_quantized_matmul_col_amd as lm
    lm.lib()
    return lm


def arguments(name, dtype):
    """Every value of the type from the smallest normal fp16 (bf16: 2^-100) to the range's end,
    both signs."""
    z = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(dtype)
    a = z.double().abs()
    return z[(a >= (2.0 ** -14 if dtype == F16 else 2.0 ** -100)) & (a <= TOP[name])]


def definition(name, z):
    """act(z), act'(z) and their bounds before the rounding to 16 bits, in 64 bits."""
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        slope = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        exponent, factor = z * z / 2, torch.zeros_like(z)
    else:
        w, factor = z, torch.ones_like(z)
        if name == "gelu_tanh":
            w, factor = TANH * (z + 0.044715 * z ** 3), TANH * (1 + 0.134145 * z * z)
        p = torch.sigmoid(w)
        slope = p * torch.sigmoid(-w) * factor
        exponent = w.abs()
    rel = 2.0 ** -19 + exponent * 2.0 ** -21
    err = rel * (p + (z * slope).abs()) + 2.0 ** -22 * z.clamp(min=0) * p * factor
    return z * p, p + z * slope, rel * (z * p).abs(), err


def held(got, want, err, z, dtype, what):
    d = (got.double() - want).abs()
    tol = fo.stored(want, err, dtype)
    bad = ~(d <= tol)
    if bool(bad.any()):
        i = int((d / tol).nan_to_num(1e30).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at z = "
                             f"{float(z[i])}: {float(got[i])} for {float(want[i])}")


@pytest.mark.parametrize("name", list(TOP))
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows", [300, None])
def test_every_argument(lm, name, dtype, rows):
    z = arguments(name, dtype)
    if rows:  # few rows: some arguments of the lower tail
        z = z[z < -2][::7][:rows]
    M, zd = z.numel(), z.double()
    act, grad, act_err, grad_err = definition(name, zd)
    X = torch.zeros((M, 8), dtype=dtype, device="cuda")
    X[:, 0], X[:, 1] = z, 1
    Wg = torch.zeros((8, 8), dtype=dtype, device="cuda")
    Wu, eye = Wg.clone(), torch.eye(8, dtype=dtype, device="cuda")
    Wg[0], Wu[1] = 1, 512
    none = torch.zeros_like(Wg)
    # products of one nonzero term: the pre-activations are the arguments themselves
    held(lm.llmint8_matmul(X, Wg, activation=name)[:, 3], act, act_err, zd, dtype, "matmul")
    # 512 times the activation: fp16 results that would be subnormal by themselves are not here
    h = lm.llmint8_gated(X, Wg, Wu, activation=name)[:, 3]
    held(h, 512 * act, 512 * act_err, zd, dtype, "gated")
    Z = z[:, None].expand(M, 8).contiguous()
    one, big = torch.ones_like(Z), torch.full_like(Z, 512)
    dX, _, _ = lm.llmint8_matmul_backward(one, None, eye, Z=Z, activation=name, need_dW=False)
    held(dX[:, 3], grad, grad_err, zd, dtype, "matmul backward")
    dU, _, _ = lm.llmint8_gated_backward(big, None, none, eye, Z, one, activation=name,
                                         need_dW=False)
    held(dU[:, 3], 512 * act, 512 * act_err, zd, dtype, "dU")
    dG, _, _ = lm.llmint8_gated_backward(one, None, eye, none, Z, big, activation=name,
                                         need_dW=False)
    held(dG[:, 3], 512 * grad, 512 * grad_err, zd, dtype, "dG")
