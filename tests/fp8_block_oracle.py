"""Block-scaled FP8 in 64 bits, from its definition in include/llmint8.h, and the bound its
product is held to.

The bound. Codes are exact, their products are exact in fp32 (two significands of 4 bits). The
MFMA adds the products of eight consecutive codes on a grid: measured, each is cut towards zero
to a multiple of 2^-13 2^(ea + eb), with the exponents of the two factors whose sum is the
largest of the eight (so computed, 83 to 94 % of random sums of 128 to 16 codes agree to 2^-22; with
groups of four or sixteen, or the exponents of the products, 5 to 55 %). So in each eight the product
p with the largest exponents is whole, since the significands' product has 6 fractional bits, and
each of the other seven loses less than 2^-13 2^(ea + eb) <= 2^-13 |p| (the significands are at
least 1: subnormal codes count by their leading bit): in all less than 7 2^-13 |p|, at most that
part of the eight's sum of magnitudes, and of all eights' together. An example: -8 beside products
of less than 0.021 loses 3.6 2^-10 = 3.5 2^-13 of the sum of magnitudes. The eights and the blocks
add to fp32 sums: K / 8 roundings at most, of 2^-23 of a partial sum each, which is at most the
sum of the magnitudes; less than K 2^-25 of it. Partial
sums of waves or parts add 16 more roundings. Then a bias and one rounding of the result."""
import torch

import ffn_oracle as fo

BLOCK = 128


def table(device):
    """The values of the 256 codes; NaN for 0x7f and 0xff."""
    c = torch.arange(256, device=device)
    m, e = (c & 7).double(), (c >> 3) & 15
    v = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(c > 127, -v, v)


def scale_bytes(top):
    """The byte of blocks with these largest magnitudes (NaN: none finite)."""
    bad = ~torch.isfinite(top)
    t = torch.where(bad, torch.ones_like(top), top)
    byte = torch.zeros_like(t, dtype=torch.int64)
    # the smallest e with top <= 448 2^e, by trying all
    for b in range(254, -1, -1):
        byte = torch.where(t <= 448 * 2.0 ** (b - 127), torch.full_like(byte, b), byte)
    return torch.where(bad, torch.full_like(byte, 255), byte)


def encode(v):
    """The codes next to v (|v| <= 448), ties to the even code."""
    t = table(v.device)[:127]  # the non-negative values in rising order
    a = v.abs().contiguous()
    hi = torch.searchsorted(t, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - t[lo], t[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return code + 128 * (torch.signbit(v)).long()


def rows(x):
    """(codes [M, K], bytes [M, blocks]) of x by blocks of 128 of a row."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    pad = torch.zeros((M, kb * BLOCK), dtype=torch.float64, device=x.device)
    pad[:, :K] = x.double()
    b = pad.view(M, kb, BLOCK)
    byte = scale_bytes(_top(b, 2))
    return _codes(b, byte[:, :, None]).view(M, -1)[:, :K].contiguous(), byte


def weights(w):
    """(codes [N, K], bytes [N blocks, K blocks]) of w [K, N] by blocks of 128 x 128."""
    K, N = w.shape
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    pad = torch.zeros((nb * BLOCK, kb * BLOCK), dtype=torch.float64, device=w.device)
    pad[:N, :K] = w.double().t()
    b = pad.view(nb, BLOCK, kb, BLOCK)
    byte = scale_bytes(_top(b, (1, 3)))
    codes = _codes(b, byte[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)
    return codes[:N, :K].contiguous(), byte


def _top(b, dims):
    t = b.abs().nan_to_num(nan=float("inf"), posinf=float("inf"))
    return t.amax(dims)


def _codes(b, byte):
    bad = byte == 255
    unit = torch.exp2((byte - 127).double())
    v = torch.where(bad, torch.zeros_like(b), b / unit)
    return torch.where(bad, torch.full_like(v, 127, dtype=torch.int64), encode(v))


def values(codes, byte_per_entry):
    """What codes stand for, given each entry's scale byte."""
    s = torch.where(byte_per_entry == 255, torch.full_like(byte_per_entry, float("nan"), dtype=torch.float64),
                    torch.exp2((byte_per_entry.long() - 127).double()))
    return table(codes.device)[codes.long()] * s


def spread_rows(byte, K):
    return byte.repeat_interleave(BLOCK, 1)[:, :K]


def spread_weights(byte, N, K):
    return byte.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def linear(x, wq, sw, bias, dtype):
    """(Y, bound) of 16-bit x with coded weights."""
    K, N = x.shape[1], wq.shape[0]
    q, byte = rows(x)
    xv = values(q, spread_rows(byte, K))
    wv = values(wq, spread_weights(sw, N, K))
    y = xv @ wv.t()
    size = xv.abs() @ wv.abs().t()
    err = (7 * 2.0 ** -13 + K * 2.0 ** -25 + 16 * 2.0 ** -23) * size
    if bias is not None:
        y = y + bias.double()
        err = err + 2.0 ** -23 * y.abs()
    return y, fo.stored(y, err, dtype)
