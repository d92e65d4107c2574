"""Measured cases of the 16-bit feed-forward operators.

  matmul           Y = act(X W + b) + R, and its backward pass (dX, dW, db)
  gated            H = act(X Wg) * (X Wu), and its backward pass (dX, dWg, dWu)
  checkpoint       a 16-bit matrix held as 8-bit codes, blocks of 32 entries of a row
                   sharing a power-of-two scale, and back

With `own` false, run() is the plain form: elementary torch operations in fp32,
rounded once at the end. With `own` true it makes the calls of the package.
"""
import math

import torch

own = False

F16, BF16 = "float16", "bfloat16"
BLOCK = 32  # entries of a row that share one checkpoint scale

# Layer sizes are those of the repository's workloads: 4096 x 11008 (7B feed-forward),
# 5120 x 13824 (13B) and 8192 x 28672 (70B); the others are generic.


def listed():
    return [
        # one token through a square projection with bias and residual: latency
        dict(name="matmul 1 token", op="matmul", M=1, K=4096, N=4096, dtype=F16, act="none",
             bias=True, residual=True),
        # a ragged chunk of a prompt through a small layer: odd rows, partial tiles on every side
        dict(name="matmul ragged 301", op="matmul", M=301, K=1040, N=520, dtype=BF16, act="gelu",
             bias=True, residual=True),
        # prompt through the 7B down projection, added to the residual stream
        dict(name="matmul 2048 down", op="matmul", M=2048, K=11008, N=4096, dtype=BF16, act="none",
             bias=False, residual=True),
        # training step of a dense layer with bias and activation
        dict(name="matmul backward 2048", op="matmul_backward", M=2048, K=4096, N=4096, dtype=BF16,
             act="gelu_tanh", bias=True, saved="full"),
        # one token through the 7B gated block: the weights are read once
        dict(name="gated 1 token", op="gated", M=1, K=4096, N=11008, dtype=F16, act="silu",
             save="none"),
        # a batch of sequences decoding through the 13B gated block
        dict(name="gated 20 tokens", op="gated", M=20, K=5120, N=13824, dtype=BF16, act="silu",
             save="none"),
        # training forward of the 13B gated block, the pre-activations kept in 8 bits
        dict(name="gated 4096 keep 8 bits", op="gated", M=4096, K=5120, N=13824, dtype=BF16,
             act="silu", save="8bit"),
        # long prompt through the 70B gated block
        dict(name="gated 8192 large", op="gated", M=8192, K=8192, N=28672, dtype=F16, act="silu",
             save="none"),
        # backward of the 7B gated block from pre-activations in 16 bits
        dict(name="gated backward 2048", op="gated_backward", M=2048, K=4096, N=11008, dtype=F16,
             act="silu", saved="full"),
        # the same from 8-bit checkpoints, a packed batch with an odd number of tokens
        dict(name="gated backward 1777 8bit", op="gated_backward", M=1777, K=4096, N=11008,
             dtype=BF16, act="gelu_tanh", saved="8bit"),
        # activations of the 13B block kept for the backward pass
        dict(name="checkpoint 4096", op="checkpoint", M=4096, K=13824, dtype=BF16),
        # a short ragged one, its last block partly filled
        dict(name="checkpoint ragged 37", op="checkpoint", M=37, K=1000, dtype=F16),
    ]


def draw(rng):
    def size(lo, hi, mult):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(mult, int(v / mult + 0.5) * mult)

    op = rng.choice(["matmul", "matmul", "matmul_backward", "gated", "gated", "gated_backward",
                     "checkpoint"])
    c = dict(op=op, dtype=rng.choice([F16, BF16]))
    if op == "checkpoint":
        c.update(M=size(1, 8192, 1), K=size(256, 28672, 8))
        return c
    # decoding batches, ragged prompts and training batches alike
    c.update(M=size(1, 4096, 1), K=size(256, 8192, 8), N=size(256, 14336, 8))
    if op in ("matmul", "matmul_backward"):
        c["act"] = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        c["bias"] = rng.random() < 0.5
    else:
        c["act"] = rng.choice(["silu", "gelu_tanh", "gelu", "relu"])
    if op == "matmul":
        c["residual"] = rng.random() < 0.5
    if op == "gated":
        c["save"] = rng.choice(["none", "full", "8bit"]) if c["M"] > 64 else "none"
    if op in ("matmul_backward", "gated_backward"):
        c["saved"] = rng.choice(["full", "8bit"])
    return c


# ---- inputs ---------------------------------------------------------------------------

def _acts(g, M, K, dtype):
    """Activations: N(0, 1) with a few feature columns 20 to 60 times larger, as the
    repository's workloads plant them."""
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.float32)
    n = max(1, K // 1024)
    cols = torch.randint(0, K, (n,), generator=g, device="cuda")
    mag = torch.rand((1, n), generator=g, device="cuda") * 40 + 20
    x[:, cols] = mag * (1 + 0.1 * x[:, cols])
    return x.to(dtype)


def _weight(g, K, N, dtype):
    return (torch.randn((K, N), generator=g, device="cuda", dtype=torch.float32) * 0.02).to(dtype)


def _grad(g, M, N, dtype):
    return (torch.randn((M, N), generator=g, device="cuda", dtype=torch.float32) * 0.1).to(dtype)


def _pre(g, M, N, dtype):
    """Pre-activations as saved by a forward pass."""
    return (torch.randn((M, N), generator=g, device="cuda", dtype=torch.float32) * 1.5).to(dtype)


def _pack(x):
    """8-bit codes (rows padded to 16 bytes) and biased exponents of a matrix."""
    M, K = x.shape
    codes, expo = _plain_pack(x)
    held = torch.zeros((M, (K + 15) // 16 * 16), dtype=torch.int8, device=x.device)
    held[:, :K] = codes.to(torch.int8)
    return held[:, :K], (expo + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, case["dtype"])
    op, M, K, N = case["op"], case["M"], case["K"], case.get("N")
    s = dict(op=op, act=case.get("act"), dtype=dt)
    s["X"] = _acts(g, M, K, dt)
    if op == "matmul":
        s["W"] = _weight(g, K, N, dt)
        s["bias"] = _pre(g, 1, N, dt)[0].contiguous() if case["bias"] else None
        s["residual"] = _acts(g, M, N, dt) if case["residual"] else None
    elif op == "matmul_backward":
        s["W"], s["dY"] = _weight(g, K, N, dt), _grad(g, M, N, dt)
        s["Z"] = _pre(g, M, N, dt) if case["act"] != "none" else None
        s["bias"] = case["bias"]
    elif op in ("gated", "gated_backward"):
        s["Wg"], s["Wu"] = _weight(g, K, N, dt), _weight(g, K, N, dt)
        s["save"] = case.get("save", "none")
        if op == "gated_backward":
            s["dH"], s["G"], s["U"] = _grad(g, M, N, dt), _pre(g, M, N, dt), _pre(g, M, N, dt)
    if case.get("saved") == "8bit":
        for k in ("X", "G", "U"):
            if k in s:
                s[k] = _pack(s[k])
    return s


# ---- plain forms ----------------------------------------------------------------------

def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        phi = torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * phi
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _blocks(x):
    """[M, K] -> [M, ceil(K / 32), 32], zeros past K."""
    M, K = x.shape
    nb = (K + BLOCK - 1) // BLOCK
    if K % BLOCK:
        pad = torch.zeros((M, nb * BLOCK), dtype=x.dtype, device=x.device)
        pad[:, :K] = x
        x = pad
    return x.view(M, nb, BLOCK)


def _pow2(e):
    """2^e as fp32 from its bits, for int32 e in [-127, 127] (2^-127 is subnormal)."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _plain_pack(x):
    """Codes [M, K] and exponents [M, ceil(K / 32)] of the blocks, in fp32."""
    M, K = x.shape
    b = _blocks(x.float())
    _, e = torch.frexp(b.abs().amax(dim=2))  # absmax = m 2^e with m in [0.5, 1)
    e = torch.clamp(e - 7, min=-127)
    e = torch.where(b.abs().amax(dim=2) > 0, e, torch.full_like(e, -127))
    codes = torch.clamp(torch.round(b * _pow2(-e)[:, :, None]), -127, 127)
    return codes.view(M, -1)[:, :K], e


def _plain_unpack(codes, e):
    M, K = codes.shape
    return (_blocks(codes.float()) * _pow2(e)[:, :, None]).view(M, -1)[:, :K]


def _value(x):
    """A saved matrix in fp32, held in 16 or 8 bits."""
    return _plain_unpack(x[0], x[1].to(torch.int32) - 127) if isinstance(x, tuple) else x.float()


def _run_plain(s):
    dt, op, act = s["dtype"], s["op"], s["act"]
    if op == "matmul":
        z = s["X"].float() @ s["W"].float()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(act, z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(dt)
    if op == "matmul_backward":
        dz = s["dY"].float()
        if act != "none":
            dz = dz * _act_grad(act, s["Z"].float())
        out = dict(dX=(dz @ s["W"].float().t()).to(dt), dW=(_value(s["X"]).t() @ dz).to(dt))
        if s["bias"]:
            out["db"] = dz.sum(dim=0)
        return out
    if op == "gated":
        x = s["X"].float()
        gate, up = x @ s["Wg"].float(), x @ s["Wu"].float()
        out = dict(H=(_act(act, gate) * up).to(dt))
        if s["save"] == "full":
            out.update(G=gate.to(dt), U=up.to(dt))
        elif s["save"] == "8bit":
            out.update(G=_plain_unpack(*_plain_pack(gate)).to(dt),
                       U=_plain_unpack(*_plain_pack(up)).to(dt))
        return out
    if op == "gated_backward":
        dh, gate, up = s["dH"].float(), _value(s["G"]), _value(s["U"])
        dg, du = dh * up * _act_grad(act, gate), dh * _act(act, gate)
        xt = _value(s["X"]).t()
        return dict(dX=(dg @ s["Wg"].float().t() + du @ s["Wu"].float().t()).to(dt),
                    dWg=(xt @ dg).to(dt), dWu=(xt @ du).to(dt))
    codes, e = _plain_pack(s["X"])
    return dict(X=_plain_unpack(codes, e).to(dt), scale=_pow2(e))


# ---- the package's calls --------------------------------------------------------------

def _run_own(s):
    import bit_quantized_matmul_col_amd as lm
    op, act = s["op"], s["act"]
    if op == "matmul":
        return lm.llmint8_matmul(s["X"], s["W"], bias=s["bias"], activation=act,
                                 residual=s["residual"])
    if op == "matmul_backward":
        dX, dW, db = lm.llmint8_matmul_backward(s["dY"], s["X"], s["W"], Z=s["Z"], activation=act,
                                                need_dbias=s["bias"])
        return dict(dX=dX, dW=dW, db=db) if s["bias"] else dict(dX=dX, dW=dW)
    if op == "gated":
        if s["save"] == "none":
            return dict(H=lm.llmint8_gated(s["X"], s["Wg"], s["Wu"], activation=act))
        H, G, U = lm.llmint8_gated(s["X"], s["Wg"], s["Wu"], activation=act, save=s["save"])
        if s["save"] == "8bit":
            G, U = (lm.llmint8_checkpoint_unpack(c, s["dtype"]) for c in (G, U))
        return dict(H=H, G=G, U=U)
    if op == "gated_backward":
        dX, dWg, dWu = lm.llmint8_gated_backward(s["dH"], s["X"], s["Wg"], s["Wu"], s["G"], s["U"],
                                                 activation=act)
        return dict(dX=dX, dWg=dWg, dWu=dWu)
    c = lm.llmint8_checkpoint_pack(s["X"])
    # the scales as the values they stand for
    return dict(X=lm.llmint8_checkpoint_unpack(c, s["dtype"]),
                scale=_pow2(c.scales.to(torch.int32) - 127))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- work and definitions -------------------------------------------------------------

def work(case):
    op, M, K, N = case["op"], case["M"], case["K"], case.get("N")
    x8, kb = 1 + 1 / BLOCK, 2  # bytes of an entry held in 8 bits; in 16 bits
    if op == "checkpoint":  # pack: 16 bits in, codes out; unpack: the reverse
        return {"bytes": 2 * M * K * (kb + x8), "flops": 4 * M * K}
    held = x8 if case.get("saved") == "8bit" else kb
    if op == "matmul":
        b = kb * (M * K + K * N + M * N * (2 if case["residual"] else 1))
        return {"bytes": b + (kb * N if case["bias"] else 0), "flops": 2 * M * K * N}
    if op == "matmul_backward":
        b = kb * (2 * K * N + M * K + M * N * (1 if case["act"] == "none" else 2)) + held * M * K
        return {"bytes": b + (4 * N if case["bias"] else 0), "flops": 4 * M * K * N}
    if op == "gated":
        save = {"none": 0, "full": 2 * kb, "8bit": 2 * x8}[case["save"]]
        return {"bytes": kb * (M * K + 2 * K * N + M * N) + save * M * N, "flops": 4 * M * K * N}
    b = kb * (M * N + 4 * K * N + M * K) + held * (M * K + 2 * M * N)
    return {"bytes": b, "flops": 8 * M * K * N}


def _sig64(z):
    return 1 / (1 + torch.exp(-z))


def _two_to(e):
    """2^e as a double with that exponent field, for int64 e in [-1022, 1023]."""
    return ((e + 1023) << 52).view(torch.float64)


def _d(x):
    """A saved matrix in 64 bits: the code times two to the exponent."""
    if not isinstance(x, tuple):
        return x.double()
    codes, scales = x
    cols = torch.arange(codes.shape[1], device=codes.device) // 32
    return codes.double() * _two_to(scales.to(torch.int64) - 127)[:, cols]


def _exact_act(name, z):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).double()
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":  # (1 + tanh(v)) / 2 is the logistic function of 2v
        k = 2 * math.sqrt(2 / math.pi)
        p = _sig64(k * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * k * (1 + 0.134145 * z ** 2)
    p = _sig64(z)
    return z * p, p + z * p * (1 - p)


def _exact_held(x):
    """What the 8-bit blocks of x stand for, in 64 bits: (values, scales)."""
    x = x.double()
    M, K = x.shape
    nb = -(-K // 32)
    full = torch.zeros((M, nb * 32), dtype=torch.float64, device=x.device)
    full[:, :K] = x
    full = full.reshape(M * nb, 32)
    top = full.abs().max(dim=1, keepdim=True).values
    # floor(log2(top)) without rounding errors: the mantissa of frexp is in [1/2, 1)
    e = torch.frexp(top).exponent.to(torch.int64) - 1 - 6
    step = _two_to(torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127))
    v = torch.round(full / step).clamp(-127, 127) * step
    return v.reshape(M, nb * 32)[:, :K], step.reshape(M, nb)


def exact(case, seed):
    s = prepare(case, seed)
    op, act = s["op"], s["act"]
    if op == "matmul":
        z = s["X"].double() @ s["W"].double()
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(act, z)[0]
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "matmul_backward":
        dz = s["dY"].double()
        if act != "none":
            dz = dz * _exact_act(act, s["Z"].double())[1]
        out = dict(dX=dz @ s["W"].double().t(), dW=_d(s["X"]).t() @ dz)
        if s["bias"]:
            out["db"] = dz.sum(dim=0)
        return out
    if op == "gated":
        x = s["X"].double()
        gate, up = x @ s["Wg"].double(), x @ s["Wu"].double()
        out = dict(H=_exact_act(act, gate)[0] * up)
        if s["save"] == "full":
            out.update(G=gate, U=up)
        elif s["save"] == "8bit":
            out.update(G=_exact_held(gate)[0], U=_exact_held(up)[0])
        return out
    if op == "gated_backward":
        dh, (a, da), up = s["dH"].double(), _exact_act(act, _d(s["G"])), _d(s["U"])
        dg, du = dh * up * da, dh * a
        x = _d(s["X"])
        dx = dg @ s["Wg"].double().t()
        dx += du @ s["Wu"].double().t()
        return dict(dX=dx, dWg=x.t() @ dg, dWu=x.t() @ du)
    v, step = _exact_held(s["X"])
    return dict(X=v, scale=step)
