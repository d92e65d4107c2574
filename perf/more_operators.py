"""Measured cases of the routed feed-forward operators and of the block-scaled FP8 product.

  route            the k experts of each token and their weights from the router's logits, the
                   expert-sorted order of the (token, expert) pairs, and the logits' gradient
  experts_gated    H_r = w_r act(x Wg_e) (x Wu_e) for every pair r = (token, expert e), in the
                   order of the experts, and its backward pass (dX, dWg, dWu, dw)
  experts_matmul   Y = sum of H_r Wd_e over a token's pairs (+ residual), and its backward
                   pass (dH, dWd)
  fp8_blocks       Y = X W + b with both in E4M3, blocks of 128 entries along the reduction
                   (X: of a row; W: of 128 columns) sharing a power-of-two scale

With `own` false, run() is the plain form: elementary torch operations in fp32 (the selection
of experts in 64 bits, so that close scores fall the same way), rounded once at the end. With
`own` true it makes the calls of the package.
"""
import math

import torch

own = False

F16, BF16, F32 = "float16", "bfloat16", "float32"
BLOCK = 128
TOP = 3.4028234663852886e38  # the largest fp32 value, which +infinity counts as

# 4096 x 11008, 5120 x 13824 and 8192 x 28672 are the feed-forward sizes of the repository's
# workloads; the experts' sizes are generic.


def listed():
    return [
        # one token chooses 8 of 64 experts: latency
        dict(name="route 1 token", op="route", M=1, E=64, k=8, dtype=F32, scores="softmax",
             renorm=True, bias=False, groups=1, top_groups=1, best=1, scale=1.0, masked=0.0),
        # a long prompt over many experts, limited to 4 of 8 groups, balanced by a bias
        dict(name="route 8192 groups", op="route", M=8192, E=256, k=8, dtype=F32,
             scores="sigmoid", renorm=True, bias=True, groups=8, top_groups=4, best=2, scale=2.5,
             masked=0.0),
        # training: the router's gradient, a padded batch with a tenth of its rows masked
        dict(name="route backward 8000", op="route_backward", M=8000, E=120, k=6, dtype=BF16,
             scores="softmax", renorm=False, scale=1.0, masked=0.1),
        # one token through its 8 experts: their weights are read once
        dict(name="experts gated 1 token", op="experts_gated", M=1, K=4096, N=1536, E=64, k=8,
             dtype=F16, act="silu", save=False),
        # training forward, unevenly loaded experts, pre-activations kept
        dict(name="experts gated 4096 keep", op="experts_gated", M=4096, K=4096, N=2048, E=32, k=4,
             dtype=BF16, act="silu", save=True),
        # its backward pass, with the weights' and the router's gradients
        dict(name="experts gated backward 4096", op="experts_gated_backward", M=4096, K=4096,
             N=2048, E=32, k=4, dtype=BF16, act="silu", masked=0.0),
        # a batch of sequences decoding: a few rows for every expert, joined and added
        dict(name="experts matmul 96 tokens", op="experts_matmul", M=96, K=5120, N=1536, E=64, k=6,
             dtype=BF16, residual=True, masked=0.0),
        # a ragged chunk of a prompt with masked rows, odd expert count, partial tiles everywhere
        dict(name="experts matmul ragged 333", op="experts_matmul", M=333, K=1040, N=520, E=11,
             k=3, dtype=F16, residual=True, masked=0.05),
        # backward of the second product of a training step, a packed odd batch
        dict(name="experts matmul backward 3001", op="experts_matmul_backward", M=3001, K=4096,
             N=2048, E=32, k=4, dtype=F16),
        # one token through the 70B up projection in FP8: half of the 16-bit weights' bytes
        dict(name="fp8 blocks 1 token", op="fp8_blocks", M=1, K=8192, N=28672, dtype=BF16,
             bias=False),
        # a ragged prompt through the 13B up projection
        dict(name="fp8 blocks 1777", op="fp8_blocks", M=1777, K=5120, N=13824, dtype=F16,
             bias=True),
        # long prompt through the 70B up projection
        dict(name="fp8 blocks 8192 large", op="fp8_blocks", M=8192, K=8192, N=28672, dtype=BF16,
             bias=False),
    ]


def draw(rng):
    def size(lo, hi, mult):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(mult, int(v / mult + 0.5) * mult)

    op = rng.choice(["route", "route", "route_backward", "experts_gated", "experts_gated",
                     "experts_gated_backward", "experts_matmul", "experts_matmul",
                     "experts_matmul_backward", "fp8_blocks", "fp8_blocks", "fp8_blocks"])
    c = dict(op=op, dtype=rng.choice([F16, BF16]))
    if op == "fp8_blocks":
        c.update(M=size(1, 4096, 1), K=size(256, 11008, 16), N=size(256, 14336, 8),
                 bias=rng.random() < 0.5)
        return c
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        E = groups * size(16 // groups, 256 // groups, 1)
        k = rng.randint(1, 8)
        c.update(M=size(1, 16384, 1), E=E, k=k, scores=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                 dtype=rng.choice([F32, F32, BF16, F16]), masked=rng.choice([0.0, 0.0, 0.1]))
        if op == "route":
            best = rng.choice([1, 2]) if groups > 1 else 1
            # enough groups for k experts
            least = -(-k // (E // groups))
            c.update(bias=rng.random() < 0.5, groups=groups, best=best,
                     top_groups=rng.randint(min(least, groups), groups))
        return c
    E = size(4, 64, 1)
    c.update(M=size(1, 4096, 1), K=size(256, 5120, 8), N=size(256, 2048, 8), E=E,
             k=rng.randint(1, min(6, E)))
    if op in ("experts_gated", "experts_gated_backward"):
        c["act"] = rng.choice(["silu", "gelu_tanh", "gelu", "relu"])
    if op == "experts_gated":
        c["save"] = c["M"] > 64 and rng.random() < 0.5
    if op == "experts_matmul":
        c["residual"] = rng.random() < 0.5
    if op in ("experts_matmul", "experts_gated_backward"):
        c["masked"] = rng.choice([0.0, 0.1])
    return c


# ---- inputs ---------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _acts(g, M, K, dtype):
    """Activations: N(0, 1) with a few feature columns 20 to 60 times larger, as the
    repository's workloads plant them."""
    x = _randn(g, M, K)
    n = max(1, K // 1024)
    cols = torch.randint(0, K, (n,), generator=g, device="cuda")
    mag = torch.rand((1, n), generator=g, device="cuda") * 40 + 20
    x[:, cols] = mag * (1 + 0.1 * x[:, cols])
    return x.to(dtype)


def _weights(g, E, K, N, dtype):
    W = torch.empty((E, K, N), dtype=dtype, device="cuda")
    for e in range(E):
        W[e] = (_randn(g, K, N) * 0.02).to(dtype)
    return W


def _logits(g, M, E, dtype, masked):
    """A router's logits: some experts more popular than others; masked rows (padding of a
    batch) hold -infinity throughout."""
    x = 1.5 * _randn(g, M, E) + _randn(g, 1, E)
    if masked:
        x[torch.rand((M,), generator=g, device="cuda") < masked] = -math.inf
    return x.to(dtype)


def _order(ids, E):
    """(offsets, order, places) of the pairs by expert: offsets [E + 1], order [M k] the pairs
    i k + j by expert and then by number, -1 behind the last; places [M, k] each pair's row in
    that order, -1 for a pair without an expert."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    key, pair = torch.sort(key, stable=True)
    offsets = (key[None, :] < torch.arange(E + 1, device=ids.device)[:, None]).sum(1)
    order = torch.where(key < E, pair, torch.full_like(pair, -1))
    places = torch.empty_like(pair)
    places[pair] = torch.where(key < E, torch.arange(pair.numel(), device=ids.device),
                               torch.full_like(pair, -1))
    return offsets.int(), order.int(), places.int().view(ids.shape)


def _fp8_weights(W):
    """E4M3 codes [N, K] and scale bytes [ceil(N / 128), ceil(K / 128)] of W [K, N]: what a
    program that serves in FP8 keeps."""
    wt = W.float().t()
    N, K = wt.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    pad = torch.zeros((nb * BLOCK, kb * BLOCK), dtype=torch.float32, device=W.device)
    pad[:N, :K] = wt
    b = pad.view(nb, BLOCK, kb, BLOCK)
    e = _exponent(b.abs().amax(dim=(1, 3)))
    codes = (b * _pow2(-e)[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:N, :K]
    return (codes.to(torch.float8_e4m3fn).contiguous().view(torch.uint8), (e + 127).to(torch.uint8))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, case["dtype"])
    op, M = case["op"], case["M"]
    s = {k: case.get(k) for k in ("op", "E", "k", "act", "save", "scores", "renorm", "groups",
                                  "top_groups", "best", "scale")}
    s["dtype"] = dt
    if op in ("route", "route_backward"):
        E, k = case["E"], case["k"]
        s["logits"] = _logits(g, M, E, dt, case["masked"])
        # what balances the load: small against the scores, of either sign
        s["bias"] = 0.1 * _randn(g, E) if case.get("bias") else None
        if op == "route_backward":
            s["ids"] = _choose(s["logits"], k, case["scores"], None, 1, 1, 1)
            s["dw"] = _randn(g, M, k)
        return s
    K, N = case["K"], case["N"]
    if op == "fp8_blocks":
        s["X"] = _acts(g, M, K, dt)
        s["Wq"], s["sw"] = _fp8_weights((_randn(g, K, N) * 0.02).to(dt))
        s["bias"] = _randn(g, N).to(dt) if case["bias"] else None
        return s
    E, k = case["E"], case["k"]
    logits = _logits(g, M, E, torch.float32, case.get("masked"))
    s["ids"] = _choose(logits, k, "softmax", None, 1, 1, 1)
    s["w"] = _mix(logits, s["ids"], "softmax", True, 1.0)
    # the order that the forward's first call made, which the later calls take
    s["plan"] = _order(s["ids"], E)
    R = M * k
    if op in ("experts_gated", "experts_gated_backward"):
        s["X"] = _acts(g, M, K, dt)
        s["Wg"], s["Wu"] = _weights(g, E, K, N, dt), _weights(g, E, K, N, dt)
        if op == "experts_gated_backward":
            s["dH"] = (_randn(g, R, N) * 0.1).to(dt)
            s["G"], s["U"] = (_randn(g, R, N) * 1.5).to(dt), (_randn(g, R, N) * 1.5).to(dt)
        return s
    s["H"] = _randn(g, R, N).to(dt)
    s["Wd"] = _weights(g, E, N, K, dt)
    if op == "experts_matmul":
        s["R"] = _acts(g, M, K, dt) if case["residual"] else None
    else:
        s["dY"] = (_randn(g, M, K) * 0.1).to(dt)
    return s


# ---- plain forms ----------------------------------------------------------------------

def _out(logits):
    """Experts that cannot be chosen: their logit is -infinity or NaN."""
    return ~(logits > -math.inf)


def _choose(logits, k, scores, bias, groups, top_groups, best):
    """ids [M, k] by falling selection value, ties to the lower index; -1 where none is left.
    The value is the score (softmax or sigmoid) plus the bias, in 64 bits; without a bias and
    with one best score for a group it is ordered by the logit, as the score is."""
    x = logits.double()
    out = _out(x)
    x = torch.clamp(x, max=TOP)
    M, E = x.shape
    if bias is None and best == 1:
        v = x
    elif scores == "softmax":
        p = torch.where(out, torch.zeros_like(x), x)
        top = torch.where(out, torch.full_like(x, -math.inf), x).amax(dim=1, keepdim=True)
        p = torch.where(out, torch.zeros_like(x), torch.exp(p - torch.clamp(top, min=-TOP)))
        v = p / torch.clamp(p.sum(dim=1, keepdim=True), min=1e-300)
    else:
        v = 1 / (1 + torch.exp(-torch.where(out, torch.zeros_like(x), x)))
    if bias is not None:
        v = v + bias.double()
    v = torch.where(out, torch.full_like(v, -math.inf), v)
    if groups > 1:
        m, _ = torch.sort(v.view(M, groups, E // groups), dim=2, descending=True)
        gv = m[:, :, 0]
        if best == 2 and E // groups > 1:
            gv = gv + torch.where(m[:, :, 1] > -math.inf, m[:, :, 1], torch.zeros_like(gv))
        _, order = torch.sort(gv, dim=1, descending=True, stable=True)
        keep = torch.zeros((M, groups), dtype=torch.bool, device=x.device)
        keep.scatter_(1, order[:, :top_groups], True)
        keep = keep[:, :, None].expand(M, groups, E // groups).reshape(M, E)
        v = torch.where(keep, v, torch.full_like(v, -math.inf))
    v, ids = torch.sort(v, dim=1, descending=True, stable=True)
    none = torch.full((), -1, dtype=torch.int32, device=x.device)
    return torch.where(v[:, :k] > -math.inf, ids[:, :k].int(), none)


def _picked(logits, ids):
    """(logits of the chosen experts, which slots hold one)"""
    x = torch.clamp(logits.float(), max=TOP)
    has = ids >= 0
    return torch.gather(x, 1, torch.clamp(ids, min=0).long()), has


def _log_sigmoid(x):
    return torch.clamp(x, max=0) - torch.log1p(torch.exp(-x.abs()))


def _mix(logits, ids, scores, renorm, scale):
    """The chosen experts' weights [M, k] in fp32, 0 where there is none."""
    c, has = _picked(logits, ids)
    c = torch.where(has, c, torch.zeros_like(c))
    if renorm:
        if scores == "sigmoid":
            c = _log_sigmoid(c)
        top = torch.where(has, c, torch.full_like(c, -math.inf)).amax(dim=1, keepdim=True)
        p = torch.where(has, torch.exp(c - torch.clamp(top, min=-TOP)), torch.zeros_like(c))
        w = p / torch.clamp(p.sum(dim=1, keepdim=True), min=1e-30)
    elif scores == "sigmoid":
        w = 1 / (1 + torch.exp(-c))
    else:
        x = torch.clamp(logits.float(), max=TOP)
        x = torch.where(_out(x), torch.full_like(x, -math.inf), x)
        top = torch.clamp(x.amax(dim=1, keepdim=True), min=-TOP)
        w = torch.exp(c - top) / torch.clamp(torch.exp(x - top).sum(dim=1, keepdim=True), min=1e-30)
    return torch.where(has, w * scale, torch.zeros_like(w))


def _route_backward(s):
    logits, ids, scale = s["logits"], s["ids"], s["scale"]
    c, has = _picked(logits, ids)
    w = _mix(logits, ids, s["scores"], s["renorm"], 1.0)
    d = torch.where(has, s["dw"] * scale, torch.zeros_like(w))
    dx = torch.zeros(logits.shape, dtype=torch.float32, device=logits.device)
    if s["scores"] == "sigmoid":
        mean = (d * w).sum(dim=1, keepdim=True) if s["renorm"] else 0
        dc = w * (d - mean) / (1 + torch.exp(torch.where(has, c, torch.zeros_like(c))))
    else:
        mean = (d * w).sum(dim=1, keepdim=True)
        dc = w * (d - mean)
        if not s["renorm"]:
            x = torch.clamp(logits.float(), max=TOP)
            x = torch.where(_out(x), torch.full_like(x, -math.inf), x)
            e = torch.exp(x - torch.clamp(x.amax(dim=1, keepdim=True), min=-TOP))
            dx = -mean * (e / torch.clamp(e.sum(dim=1, keepdim=True), min=1e-30))
            dc = w * d
    # the slots without an expert add nothing
    dx = dx.scatter_add(1, torch.clamp(ids, min=0).long(),
                        torch.where(has, dc, torch.zeros_like(dc)))
    return dx.to(logits.dtype)


def _act(name, z):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _act_grad(name, z):
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


def _runs(offsets):
    """(expert, first row, end) of the experts that have rows."""
    at = offsets.tolist()
    return [(e, at[e], at[e + 1]) for e in range(len(at) - 1) if at[e + 1] > at[e]]


def _plain_gated(s):
    offsets, order, _ = _order(s["ids"], s["E"])
    X, Wg, Wu, k = s["X"].float(), s["Wg"], s["Wu"], s["k"]
    R, N = order.numel(), Wg.shape[2]
    H, G, U = (torch.empty((R, N), dtype=s["dtype"], device=X.device) for _ in range(3))
    w = s["w"].reshape(-1)
    for e, a, b in _runs(offsets):
        pair = order[a:b].long()
        x = X[pair // k]
        gate, up = x @ Wg[e].float(), x @ Wu[e].float()
        H[a:b] = (w[pair][:, None] * _act(s["act"], gate) * up).to(s["dtype"])
        if s["save"]:
            G[a:b], U[a:b] = gate.to(s["dtype"]), up.to(s["dtype"])
    return dict(H=H, G=G, U=U) if s["save"] else dict(H=H)


def _plain_gated_backward(s):
    (offsets, order, _), k, dt = s["plan"], s["k"], s["dtype"]
    X, Wg, Wu = s["X"].float(), s["Wg"], s["Wu"]
    dX = torch.zeros_like(X)
    dWg, dWu = torch.zeros_like(Wg), torch.zeros_like(Wu)
    w = s["w"].reshape(-1)
    dw = torch.zeros_like(w)
    for e, a, b in _runs(offsets):
        pair = order[a:b].long()
        x, we = X[pair // k], w[pair][:, None]
        d, gate, up = s["dH"][a:b].float(), s["G"][a:b].float(), s["U"][a:b].float()
        act = _act(s["act"], gate)
        dw[pair] = (d * act * up).sum(dim=1)
        dg, du = we * d * up * _act_grad(s["act"], gate), we * d * act
        dX.index_add_(0, pair // k, dg @ Wg[e].float().t() + du @ Wu[e].float().t())
        dWg[e], dWu[e] = (x.t() @ dg).to(dt), (x.t() @ du).to(dt)
    return dict(dX=dX.to(dt), dWg=dWg, dWu=dWu, dw=dw.view(s["w"].shape))


def _plain_matmul(s):
    (offsets, order, _), k = s["plan"], s["k"]
    H, Wd = s["H"], s["Wd"]
    Y = torch.zeros((order.numel() // k, Wd.shape[2]), dtype=torch.float32, device=H.device)
    if s["R"] is not None:
        Y += s["R"].float()
    for e, a, b in _runs(offsets):
        Y.index_add_(0, order[a:b].long() // k, H[a:b].float() @ Wd[e].float())
    return Y.to(s["dtype"])


def _plain_matmul_backward(s):
    (offsets, order, _), k = s["plan"], s["k"]
    H, Wd, dY = s["H"], s["Wd"], s["dY"].float()
    dH, dWd = torch.empty_like(H), torch.zeros_like(Wd)
    for e, a, b in _runs(offsets):
        d = dY[order[a:b].long() // k]
        dH[a:b] = (d @ Wd[e].float().t()).to(s["dtype"])
        dWd[e] = (H[a:b].float().t() @ d).to(s["dtype"])
    return dict(dH=dH, dWd=dWd)


def _exponent(top):
    """int32 e of blocks with these largest magnitudes: the smallest with top <= 448 2^e, at
    least -127 (there for a block of zeros)."""
    m, e = torch.frexp(top)  # top = m 2^e with m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(top > 0, torch.clamp(e, min=-127), torch.full_like(e, -127))


def _pow2(e):
    """2^e as fp32 from its bits, for int32 e in [-127, 127] (2^-127 is subnormal)."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _plain_fp8(s):
    X, Wq, sw = s["X"].float(), s["Wq"], s["sw"]
    M, K = X.shape
    N, kb = Wq.shape[0], sw.shape[1]
    pad = torch.zeros((M, kb * BLOCK), dtype=torch.float32, device=X.device)
    pad[:, :K] = X
    b = pad.view(M, kb, BLOCK)
    e = _exponent(b.abs().amax(dim=2))
    q = (b * _pow2(-e)[:, :, None]).to(torch.float8_e4m3fn).float() * _pow2(e)[:, :, None]
    w = Wq.view(torch.float8_e4m3fn).float()
    scale = _pow2(sw.int() - 127).repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    y = q.view(M, -1)[:, :K] @ (w * scale).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["dtype"])


def _run_plain(s):
    op = s["op"]
    if op == "route":
        ids = _choose(s["logits"], s["k"], s["scores"], s["bias"], s["groups"], s["top_groups"],
                      s["best"])
        offsets, order, places = _order(ids, s["E"])
        return dict(ids=ids, weights=_mix(s["logits"], ids, s["scores"], s["renorm"], s["scale"]),
                    offsets=offsets, order=order, places=places)
    return {"route_backward": _route_backward, "experts_gated": _plain_gated,
            "experts_gated_backward": _plain_gated_backward, "experts_matmul": _plain_matmul,
            "experts_matmul_backward": _plain_matmul_backward, "fp8_blocks": _plain_fp8}[op](s)


# ---- the package's calls --------------------------------------------------------------

def _run_own(s):
    import bit_quantized_matmul_col_amd as lm
    op = s["op"]
    if op == "route":
        ids, w = lm.llmint8_route(s["logits"], s["k"], scores=s["scores"], bias=s["bias"],
                                  groups=s["groups"], top_groups=s["top_groups"],
                                  group_best=s["best"], renormalize=s["renorm"], scale=s["scale"])
        plan = lm.llmint8_expert_plan(ids, s["E"])
        return dict(ids=ids, weights=w, offsets=plan.offsets, order=plan.order, places=plan.places)
    if op == "route_backward":
        return lm.llmint8_route_backward(s["dw"], s["logits"], s["ids"], scores=s["scores"],
                                         renormalize=s["renorm"], scale=s["scale"])
    if op == "fp8_blocks":
        return lm.llmint8_linear_blockwise_fp8(s["X"], s["Wq"], s["sw"], bias=s["bias"])
    if op == "experts_gated":
        plan = lm.llmint8_expert_plan(s["ids"], s["E"])
        out = lm.llmint8_experts_gated(s["X"], s["Wg"], s["Wu"], plan, weights=s["w"],
                                       activation=s["act"], save="full" if s["save"] else "none")
        return dict(zip("HGU", out)) if s["save"] else dict(H=out)
    plan = lm.ExpertPlan(*s["plan"])
    if op == "experts_gated_backward":
        dX, dWg, dWu, dw = lm.llmint8_experts_gated_backward(
            s["dH"], s["X"], s["Wg"], s["Wu"], s["G"], s["U"], plan, weights=s["w"],
            activation=s["act"])
        return dict(dX=dX, dWg=dWg, dWu=dWu, dw=dw)
    if op == "experts_matmul":
        return lm.llmint8_experts_matmul(s["H"], s["Wd"], plan, residual=s["R"])
    dH, dWd = lm.llmint8_experts_matmul_backward(s["dY"], s["H"], s["Wd"], plan)
    return dict(dH=dH, dWd=dWd)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- work and definitions -------------------------------------------------------------

def work(case):
    op, M = case["op"], case["M"]
    if op in ("route", "route_backward"):
        E, k, size = case["E"], case["k"], 4 if case["dtype"] == F32 else 2
        if op == "route":  # logits; ids, weights, order and places; a few operations a score
            return {"bytes": M * E * size + 16 * M * k + 4 * E, "flops": 8 * M * E}
        return {"bytes": 2 * M * E * size + 8 * M * k, "flops": 8 * M * E}
    K, N = case["K"], case["N"]
    if op == "fp8_blocks":
        codes = 1 + 1 / BLOCK ** 2
        return {"bytes": 2 * M * K + codes * K * N + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * K * N}
    E, k = case["E"], case["k"]
    R = M * k * (1 - case.get("masked", 0.0))
    # experts that get a token, were each token's choice uniform; every expert's gradient
    used = E * (1 - (1 - k / E) ** M)
    if op == "experts_gated":
        b = 2 * (M * K + 2 * used * K * N + R * N * (3 if case["save"] else 1)) + 8 * M * k
        return {"bytes": b, "flops": 4 * R * K * N}
    if op == "experts_gated_backward":
        b = 2 * (2 * M * K + 2 * (used + E) * K * N + 3 * R * N) + 12 * M * k
        return {"bytes": b, "flops": 8 * R * K * N}
    if op == "experts_matmul":
        b = 2 * (R * N + used * K * N + M * K * (2 if case["residual"] else 1)) + 4 * M * k
        return {"bytes": b, "flops": 2 * R * K * N}
    b = 2 * (M * K + 2 * R * N + (used + E) * K * N) + 4 * M * k
    return {"bytes": b, "flops": 4 * R * K * N}


def _sig64(z):
    return torch.where(z >= 0, 1 / (1 + torch.exp(-z.abs())),
                       torch.exp(-z.abs()) / (1 + torch.exp(-z.abs())))


def _exact_act(name, z):
    """(act(z), act'(z)) in 64 bits."""
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


def _exact_scores(s):
    """(scores of all experts, 0 where masked; which experts are masked), in 64 bits."""
    x = s["logits"].double()
    dead = torch.isnan(x) | torch.isneginf(x)
    x = x.masked_fill(dead, 0).clamp(max=TOP)
    if s["scores"] == "sigmoid":
        return _sig64(x).masked_fill(dead, 0), dead, x
    x = x.masked_fill(dead, -math.inf)
    full = dead.all(dim=1, keepdim=True)
    p = torch.softmax(x.masked_fill(full, 0), dim=1)
    return p.masked_fill(dead, 0), dead, x.masked_fill(dead, 0)


def _exact_route(s):
    p, dead, x = _exact_scores(s)
    M, E = p.shape
    k, groups = s["k"], s["groups"]
    v = x.clone() if s["bias"] is None and s["best"] == 1 else p.clone()
    if s["bias"] is not None:
        v += s["bias"].double()
    v[dead] = -math.inf
    each = E // groups
    if groups > 1:
        # a group's value is its highest, or the sum of its two highest
        part = v.view(M, groups, each).clone()
        gv = part.max(dim=2).values
        if s["best"] == 2 and each > 1:
            part.scatter_(2, part.argmax(dim=2, keepdim=True), -math.inf)
            second = part.max(dim=2).values
            gv = gv + second.masked_fill(torch.isinf(second), 0)
        # groups that beat this one, or tie with it from a lower index
        low = torch.ones((groups, groups), dtype=torch.bool, device=v.device).tril(-1)
        beats = (gv[:, None, :] > gv[:, :, None]) | ((gv[:, None, :] == gv[:, :, None]) & low)
        drop = beats.sum(dim=2) >= s["top_groups"]
        v[drop.repeat_interleave(each, dim=1)] = -math.inf
    ids = torch.full((M, k), -1, dtype=torch.int32, device=v.device)
    w = torch.zeros((M, k), dtype=torch.float64, device=v.device)
    rows = torch.arange(M, device=v.device)
    index = torch.arange(E, device=v.device)
    picked = torch.full((M, k), -math.inf, dtype=torch.float64, device=v.device)
    for j in range(min(k, E)):
        top = v.max(dim=1).values
        first = torch.where(v == top[:, None], index, torch.full_like(index, E)).min(dim=1).values
        live = top > -math.inf
        first = first.clamp(max=E - 1)
        ids[:, j] = torch.where(live, first, torch.full_like(first, -1)).int()
        w[:, j] = torch.where(live, p[rows, first], torch.zeros_like(top))
        picked[:, j] = torch.where(live, x[rows, first], picked[:, j])
        v[rows, first] = -math.inf
    if s["renorm"]:
        live = ids >= 0
        if s["scores"] == "softmax":
            z = picked
        else:  # log of the logistic function
            z = torch.where(live, -torch.log1p(torch.exp(-picked.clamp(min=-300))), picked)
        empty = ~live.any(dim=1, keepdim=True)
        w = torch.softmax(z.masked_fill(empty, 0), dim=1).masked_fill(~live, 0)
    counts = torch.bincount(ids[ids >= 0].long(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    flat = ids.view(-1)
    live = (flat >= 0).nonzero().view(-1)
    order = torch.full_like(flat, -1)
    # a key that no two pairs share, so any sort gives the one order
    key = flat[live].long() * flat.numel() + live
    order[:live.numel()] = live[key.argsort()].int()
    places = torch.full_like(flat, -1)
    places[order[:live.numel()].long()] = torch.arange(live.numel(), device=v.device).int()
    return dict(ids=ids, weights=w * s["scale"], offsets=offsets.int(), order=order,
                places=places.view(M, k))


def _exact_route_backward(s):
    p, dead, x = _exact_scores(s)
    M, E = p.shape
    ids, k = s["ids"], s["k"]
    # which slot each expert has, as a 0/1 matrix [M, k, E]
    hot = (ids[:, :, None] == torch.arange(E, device=ids.device)).double()
    d = torch.bmm((s["dw"].double() * s["scale"])[:, None, :], hot)[:, 0]
    chosen = hot.sum(dim=1)
    if s["scores"] == "softmax":
        if s["renorm"]:
            z = torch.where(chosen > 0, x, torch.full_like(x, -math.inf))
            empty = (chosen == 0).all(dim=1, keepdim=True)
            p = torch.softmax(z.masked_fill(empty, 0), dim=1) * chosen
        return p * (d - (p * d).sum(dim=1, keepdim=True))
    slope = _sig64(x) * _sig64(-x) * chosen
    if not s["renorm"]:
        return d * slope
    total = (p * chosen).sum(dim=1, keepdim=True)
    total = total.masked_fill(total == 0, 1)
    mean = (d * p * chosen).sum(dim=1, keepdim=True) / total
    return slope * (d - mean) / total


def _exact_experts(s):
    op, k, E = s["op"], s["k"], s["E"]
    ids = s["ids"]
    flat = ids.reshape(-1)
    # rows by expert, pair by pair within one
    pairs = [(flat == e).nonzero().view(-1) for e in range(E)]
    at, out = 0, {}
    M, dev = ids.shape[0], ids.device
    R = flat.numel()
    f64 = dict(dtype=torch.float64, device=dev)
    if op == "experts_gated":
        N = s["Wg"].shape[2]
        out = {n: torch.zeros((R, N), **f64) for n in ("HGU" if s["save"] else "H")}
    elif op == "experts_matmul":
        Y = torch.zeros((M, s["Wd"].shape[2]), **f64) if s["R"] is None else s["R"].double()
    elif op == "experts_matmul_backward":
        out = dict(dH=torch.zeros(s["H"].shape, **f64), dWd=torch.zeros(s["Wd"].shape, **f64))
    else:
        out = dict(dX=torch.zeros(s["X"].shape, **f64), dWg=torch.zeros(s["Wg"].shape, **f64),
                   dWu=torch.zeros(s["Wu"].shape, **f64), dw=torch.zeros((R,), **f64))
    for e, p in enumerate(pairs):
        n = p.numel()
        if n == 0:
            continue
        rows, token = slice(at, at + n), p // k
        at += n
        if op == "experts_matmul":
            y = s["H"][rows].double() @ s["Wd"][e].double()
            Y.index_add_(0, token, y)
        elif op == "experts_matmul_backward":
            d = s["dY"].double()[token]
            out["dH"][rows] = torch.matmul(d, s["Wd"][e].double().t())
            out["dWd"][e] = torch.matmul(s["H"][rows].double().t(), d)
        else:
            x, w = s["X"][token].double(), s["w"].reshape(-1)[p].double().unsqueeze(1)
            wg, wu = s["Wg"][e].double(), s["Wu"][e].double()
            if op == "experts_gated":
                gate, up = x @ wg, x @ wu
                out["H"][rows] = _exact_act(s["act"], gate)[0] * up * w
                if s["save"]:
                    out["G"][rows], out["U"][rows] = gate, up
                continue
            a, da = _exact_act(s["act"], s["G"][rows].double())
            up, d = s["U"][rows].double(), s["dH"][rows].double()
            out["dw"][p] = (d * (a * up)).sum(dim=1)
            dg, du = (d * w) * (up * da), (d * w) * a
            out["dX"].index_add_(0, token, dg @ wg.t() + du @ wu.t())
            out["dWg"][e], out["dWu"][e] = x.t() @ dg, x.t() @ du
    if op == "experts_matmul":
        return Y
    if "dw" in out:
        out["dw"] = out["dw"].view(ids.shape)
    return out


def _e4m3(v):
    """The E4M3 value next to v (|v| <= 448), ties to even, in 64 bits."""
    e = torch.frexp(v).exponent.clamp(min=-5) - 1  # 2^e <= |v| < 2^(e + 1), at least 2^-6
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return torch.round(v / step) * step


def _exact_fp8(s):
    x, (M, K) = s["X"].double(), s["X"].shape
    value = torch.empty_like(x)
    for c in range(0, K, 128):
        b = x[:, c:c + 128]
        top = b.abs().max(dim=1, keepdim=True).values
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448))
        # the logarithm may be off by an ulp next to an integer
        e = e + (top > 448 * torch.exp2(e)).double() - (top <= 448 * torch.exp2(e - 1)).double()
        unit = torch.exp2(e.clamp(min=-127))
        value[:, c:c + 128] = _e4m3(b / unit) * unit
    code = torch.arange(256, device=x.device)
    mant, expo = (code & 7).double(), (code >> 3) & 15
    table = torch.where(expo > 0, (8 + mant) * torch.exp2(expo.double() - 10), mant * 2.0 ** -9)
    table = torch.where(code > 127, -table, table)
    Wq, sw = s["Wq"], s["sw"]
    N = Wq.shape[0]
    y = torch.empty((M, N), dtype=torch.float64, device=x.device)
    for r in range(0, N, 128):
        w = table[Wq[r:r + 128].long()]
        unit = torch.exp2(sw[r // 128].double() - 127)
        w *= unit[torch.arange(K, device=x.device) // 128]
        y[:, r:r + 128] = value @ w.t()
    return y if s["bias"] is None else y + s["bias"].double()


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        return _exact_route(s)
    if s["op"] == "route_backward":
        return _exact_route_backward(s)
    return _exact_fp8(s) if s["op"] == "fp8_blocks" else _exact_experts(s)
