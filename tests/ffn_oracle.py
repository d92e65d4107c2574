"""The 16-bit feed-forward operators in 64 bits (torch, CPU or GPU), from their
definitions in include/llmint8.h, with the error bounds the kernels are held to.

Bounds, for inputs taken as exact. u is the unit roundoff of the result's type
(2^-11 fp16, 2^-8 bf16), tiny half its smallest subnormal.
  * A sum of K products in fp32: every addition rounds (or truncates) by at most
    2^-23 of a partial sum; partial sums are of the size of the root of the sum of
    the squared products, r. K 2^-23 r bounds what K such roundings add up to.
  * A rounding of the result: u |result| + tiny.
  * A product whose operand was rounded to 16 bits first (dZ, dG, dU): independent
    errors of at most u per term add up to less than 4 u r (7 standard deviations),
    and subnormal operands to at most tiny times the sum of the other's magnitudes.
  * An activation in fp32: 2^-20 of max(|z|, 1), several times its few roundings,
    and its slope, at most 1.13 (gelu), times the error of its argument.
"""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
SLOPE = 1.13


def act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return (0.5 * torch.special.erfc(-z / math.sqrt(2))
                + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return (1 + t) / 2 + z * (1 - t * t) / 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def product(a, b):
    """a b and the bound on its fp32 sum."""
    return a @ b, a.shape[1] * 2.0 ** -23 * root(a, b)


def root(a, b):
    return torch.sqrt((a * a) @ (b * b))


def act_err(z, dz):
    return SLOPE * dz + 2.0 ** -20 * torch.clamp(z.abs(), min=1)


def stored(y, err, dtype):
    return err + U[dtype] * (y.abs() + err) + TINY[dtype]


def matmul(X, W, bias, residual, name, dtype):
    """((Y, bound), (Z, bound))"""
    z, dz = product(X, W)
    if bias is not None:
        z = z + bias
        dz = dz + 2.0 ** -23 * z.abs()
    y = act(name, z)
    dy = dz if name == "none" else act_err(z, dz)
    if residual is not None:
        y = y + residual
        dy = dy + 2.0 ** -23 * y.abs()
    return (y, stored(y, dy, dtype)), (z, stored(z, dz, dtype))


def gated(X, Wg, Wu, name, dtype):
    """((H, bound), (G, bound), (U, bound)); the last two before any rounding."""
    g, dg = product(X, Wg)
    u, du = product(X, Wu)
    a, da = act(name, g), act_err(g, dg)
    h = a * u
    dh = da * u.abs() + a.abs() * du + da * du
    return (h, stored(h, dh, dtype)), (g, dg), (u, du)


def rounded_product(a, b, da, rounded_a, dtype):
    """a b where one factor (a if rounded_a) carries an error da and a rounding."""
    y, err = product(a, b)
    other = b if rounded_a else a
    small = TINY[dtype] * (other.abs().sum(0)[None, :] if rounded_a
                           else other.abs().sum(1)[:, None])
    err = err + 4 * U[dtype] * root(a, b) + small
    err = err + (da @ b.abs() if rounded_a else a.abs() @ da)
    return y, err


def matmul_backward(dY, X, W, Z, name, dtype, act_none_rounds=False):
    """((dX, bound), (dW, bound), (db, bound))"""
    if name == "none":
        dz, e = dY, torch.zeros_like(dY)
    else:
        dz = dY * act_grad(name, Z)
        e = dY.abs() * 2.0 ** -19 * torch.clamp(Z.abs(), min=1)
    x, ex = rounded_product(dz, W.t(), e, True, dtype)
    w, ew = rounded_product(X.t(), dz, e, False, dtype)
    db = dz.sum(0)
    edb = dz.shape[0] * 2.0 ** -23 * torch.sqrt((dz * dz).sum(0)) + e.sum(0)
    return (x, stored(x, ex, dtype)), (w, stored(w, ew, dtype)), (db, edb + 2.0 ** -140)


def gated_backward(dH, X, Wg, Wu, G, U_, name, dtype):
    """((dX, bound), (dWg, bound), (dWu, bound))"""
    dg, du = dH * U_ * act_grad(name, G), dH * act(name, G)
    top = torch.clamp(G.abs(), min=1)
    eg, eu = (dH * U_).abs() * 2.0 ** -19 * top, dH.abs() * 2.0 ** -20 * top
    x1, e1 = rounded_product(dg, Wg.t(), eg, True, dtype)
    x2, e2 = rounded_product(du, Wu.t(), eu, True, dtype)
    wg, e3 = rounded_product(X.t(), dg, eg, False, dtype)
    wu, e4 = rounded_product(X.t(), du, eu, False, dtype)
    x = x1 + x2
    # one sum of twice the length
    ex = 2 * (e1 + e2)
    return (x, stored(x, ex, dtype)), (wg, stored(wg, e3, dtype)), (wu, stored(wu, e4, dtype))


def pack(x):
    """(codes, scale bytes) of the 8-bit checkpoint of x, by the format's definition."""
    x = x.double()
    M, K = x.shape
    nb = -(-K // 32)
    b = torch.zeros((M, nb * 32), dtype=torch.float64, device=x.device)
    b[:, :K] = x
    b = b.view(M, nb, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    top = torch.where(bad, torch.ones_like(top), top)
    e = torch.frexp(top)[1].long() - 1 - 6
    e = torch.clamp(torch.where(top > 0, e, torch.full_like(e, -127)), min=-127)
    codes = torch.clamp(torch.round(b / pow2(e)[:, :, None]), -127, 127)
    codes = torch.where(bad[:, :, None], torch.zeros_like(codes), codes)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127)
    return codes.view(M, nb * 32)[:, :K].to(torch.int8), byte.to(torch.uint8)


def pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def unpack(codes, byte):
    K = codes.shape[1]
    s = torch.where(byte == 255, torch.full_like(byte, float("nan"), dtype=torch.float64),
                    pow2(byte.long() - 127))
    return codes.double() * s.repeat_interleave(32, dim=1)[:, :K]
