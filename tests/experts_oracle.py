"""The routed feed-forward operators in 64 bits (torch, CPU or GPU), from their definitions in
include/llmint8.h, with the error bounds the kernels are held to (ffn_oracle.py has the rules
for sums, roundings and activations).

Further bounds, with eps = 2^-23 and the fp32 exponential, logarithm and division good to a few
units in the last place:
  * exp(x - top) has the relative error |x - top| eps from its argument and a few eps of its own;
    a sum over E of them adds at most E eps, a quotient one more. So a weight is good to
    (2 r + E + 16) eps of itself, r the largest |x - top| whose term counts, and to the smallest
    normal number where it is below that.
  * a sum over a token's k rows in fp32 adds k eps of the sum of their magnitudes; rows that were
    stored in 16 bits first add a rounding each.
"""
import math

import torch

import ffn_oracle as fo

EPS = 2.0 ** -23
TOP = 3.4028234663852886e38
SMALL = 2.0 ** -126


def choose_row(x, k, scores, bias, groups, top_groups, best):
    """The ids of one row (a list of floats), by sorting."""
    E = len(x)
    live = [v > -math.inf for v in x]
    x = [min(v, TOP) if ok else 0.0 for v, ok in zip(x, live)]
    if bias is None and (best == 1 or groups == 1):
        val = list(x)
    elif scores == "sigmoid":
        val = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in x]
    else:
        top = max([v for v, ok in zip(x, live) if ok], default=0.0)
        e = [math.exp(v - top) if ok else 0.0 for v, ok in zip(x, live)]
        val = [v / max(math.fsum(e), 1e-300) for v in e]
    if bias is not None:
        val = [v + b for v, b in zip(val, bias)]
    val = [v if ok else -math.inf for v, ok in zip(val, live)]
    each = E // groups
    if groups > 1:
        score = []
        for g in range(groups):
            top = sorted(val[g * each:(g + 1) * each], reverse=True)[:best]
            top = [v for v in top if v > -math.inf]
            score.append(sum(top) if top else -math.inf)
        order = sorted(range(groups), key=lambda g: (-score[g], g))[:top_groups]
        val = [v if i // each in order else -math.inf for i, v in enumerate(val)]
    order = sorted(range(E), key=lambda i: (-val[i], i))[:k]
    return [i if val[i] > -math.inf else -1 for i in order]


def choose(logits, k, scores="softmax", bias=None, groups=1, top_groups=1, best=1):
    b = None if bias is None else bias.double().cpu().tolist()
    rows = [choose_row(r, k, scores, b, groups, top_groups, best)
            for r in logits.double().cpu().tolist()]
    return torch.tensor(rows, dtype=torch.int32, device=logits.device)


def _clean(logits):
    """(logits with masked ones as -inf and infinities clamped, which are masked)"""
    x = logits.double()
    dead = ~(x > -math.inf)
    return torch.where(dead, torch.full_like(x, -math.inf), x.clamp(max=TOP)), dead


def slots(logits, ids):
    """(chosen logits, -inf in a slot without one; which slots have one)"""
    x, _ = _clean(logits)
    c = torch.gather(x, 1, ids.clamp(min=0, max=x.shape[1] - 1).long())
    has = (ids >= 0) & (ids < x.shape[1]) & (c > -math.inf)
    return torch.where(has, c, torch.full_like(c, -math.inf)), has


def log_sigmoid(c):
    return -torch.log1p(torch.exp(-c.abs())) + c.clamp(max=0)


def _softmax(z, over):
    """Softmax of z over the entries of `over`, zeros where there are none, and the largest
    distance to the top among the terms that count."""
    top = torch.where(over, z, torch.full_like(z, -TOP)).amax(1, keepdim=True)
    e = torch.where(over, torch.exp(torch.where(over, z - top, torch.zeros_like(z))),
                    torch.zeros_like(z))
    far = torch.where(over & (e > 1e-40), top - z, torch.zeros_like(z)).amax(1, keepdim=True)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300), far


def mix(logits, ids, scores, renorm):
    """(weights before the scale, bound), 0 in empty slots."""
    x, dead = _clean(logits)
    c, has = slots(logits, ids)
    E = x.shape[1]
    zero = torch.zeros_like(c)
    if renorm:
        z = torch.where(has, c, zero)
        if scores == "sigmoid":
            z = log_sigmoid(z)
        w, far = _softmax(z, has)
        return w, w * (4 * far + E + 32) * EPS + SMALL
    if scores == "sigmoid":
        w = torch.where(has, torch.sigmoid(torch.where(has, c, zero)), zero)
        return w, w * (c.clamp(min=-200, max=200).abs().nan_to_num() + 16) * EPS + SMALL
    p, far = _softmax(torch.where(dead, torch.zeros_like(x), x), ~dead)
    w = torch.where(has, torch.gather(p, 1, ids.clamp(min=0, max=E - 1).long()), zero)
    return w, w * (2 * far + E + 16) * EPS + SMALL


def route_backward(dw, logits, ids, scores, renorm, scale):
    """(dlogits, bound before the rounding to the logits' type)"""
    x, dead = _clean(logits)
    c, has = slots(logits, ids)
    w, ew = mix(logits, ids, scores, renorm)
    zero = torch.zeros_like(w)
    d = torch.where(has, dw.double() * scale, zero)
    E = x.shape[1]
    mean = (w * d).sum(1, keepdim=True) if renorm or scores == "softmax" else 0 * d[:, :1]
    emean = (ew * d.abs() + 40 * EPS * (w * d).abs()).sum(1, keepdim=True)
    dx, ex = torch.zeros_like(x), torch.zeros_like(x)
    if scores == "sigmoid":
        s = torch.where(has, torch.sigmoid(-torch.where(has, c, zero)), zero)
        es = s * (c.clamp(min=-200, max=200).abs() + 16) * EPS + SMALL
        g = w * s * (d - mean)
        eg = (d.abs() + mean.abs()) * (ew * s + w * es + 8 * EPS * w * s) + w * s * emean
    elif renorm:
        g = w * (d - mean)
        eg = (d.abs() + mean.abs()) * (ew + 8 * EPS * w) + w * emean
    else:
        g, eg = w * d, ew * d.abs() + 8 * EPS * (w * d).abs()
        p, far = _softmax(torch.where(dead, torch.zeros_like(x), x), ~dead)
        dx = -mean * p
        ex = p * emean + mean.abs() * p * (2 * far + E + 24) * EPS
    at = ids.clamp(min=0, max=E - 1).long()
    dx = dx.scatter_add(1, at, torch.where(has, g, zero))
    ex = ex.scatter_add(1, at, torch.where(has, eg + 8 * EPS * g.abs(), zero))
    return dx, ex + 4 * EPS * dx.abs() + SMALL


def plan(ids, E):
    """(offsets, order, places) by going through the pairs."""
    flat = ids.reshape(-1).cpu().tolist()
    lists = [[p for p, e in enumerate(flat) if e == x] for x in range(E)]
    offsets, order = [0], []
    for one in lists:
        order += one
        offsets.append(len(order))
    places = [-1] * len(flat)
    for r, p in enumerate(order):
        places[p] = r
    order += [-1] * (len(flat) - len(order))
    as_t = lambda v: torch.tensor(v, dtype=torch.int32, device=ids.device)  # noqa: E731
    return as_t(offsets), as_t(order), as_t(places).view(ids.shape)


def runs(p, k):
    """(expert, its rows, its pairs, its tokens) of the experts that have rows."""
    at = p[0].tolist()
    for e in range(len(at) - 1):
        if at[e + 1] > at[e]:
            pair = p[1][at[e]:at[e + 1]].long()
            yield e, slice(at[e], at[e + 1]), pair, pair // k


def gated(X, Wg, Wu, p, w, name, dtype):
    """{"H", "G", "U"}: (values, bound) [M k, N], zeros behind the last row."""
    k, N = p[2].shape[1], Wg.shape[2]
    out = {n: tuple(torch.zeros((p[1].numel(), N), dtype=torch.float64, device=X.device)
                    for _ in range(2)) for n in "HGU"}
    for e, rows, pair, token in runs(p, k):
        g, dg = fo.product(X[token], Wg[e])
        u, du = fo.product(X[token], Wu[e])
        wr = torch.ones_like(g[:, :1]) if w is None else w.reshape(-1)[pair].double()[:, None]
        a, da = fo.act(name, g), fo.act_err(g, dg)
        h = wr * a * u
        dh = wr.abs() * (da * u.abs() + a.abs() * du + da * du) + 2 * EPS * h.abs()
        for n, v, dv in (("H", h, dh), ("G", g, dg), ("U", u, du)):
            out[n][0][rows], out[n][1][rows] = v, fo.stored(v, dv, dtype)
    return out


def matmul(H, Wd, p, residual, dtype, rounded):
    """(Y, bound); rounded: the rows go through 16 bits before they are summed."""
    M, k = p[2].shape
    y = torch.zeros((M, Wd.shape[2]), dtype=torch.float64, device=H.device)
    err, size = torch.zeros_like(y), torch.zeros_like(y)
    if residual is not None:
        y, size = y + residual, residual.abs()
    for e, rows, _, token in runs(p, k):
        v, dv = fo.product(H[rows], Wd[e])
        if rounded:
            dv = fo.stored(v, dv, dtype)
        y.index_add_(0, token, v), err.index_add_(0, token, dv), size.index_add_(0, token, v.abs())
    return y, fo.stored(y, err + k * EPS * size, dtype)


def matmul_backward(dY, H, Wd, p, dtype):
    """{"dH", "dWd"}: (values, bound)"""
    k = p[2].shape[1]
    dH = tuple(torch.zeros_like(H) for _ in range(2))
    dW = tuple(torch.zeros_like(Wd) for _ in range(2))
    for e, rows, _, token in runs(p, k):
        for (v, dv), to, at in ((fo.product(dY[token], Wd[e].t()), dH, rows),
                                (fo.product(H[rows].t(), dY[token]), dW, e)):
            to[0][at], to[1][at] = v, fo.stored(v, dv, dtype)
    return dict(dH=dH, dWd=dW)


def gated_backward(dH, X, Wg, Wu, G, U, p, w, name, dtype):
    """{"dX", "dWg", "dWu", "dw"}: (values, bound)"""
    M, k = p[2].shape
    zeros = lambda t: tuple(torch.zeros_like(t) for _ in range(2))  # noqa: E731
    dX, dWg, dWu = zeros(X), zeros(Wg), zeros(Wu)
    dw = tuple(torch.zeros((M * k,), dtype=torch.float64, device=X.device) for _ in range(2))
    size = torch.zeros_like(X)
    for e, rows, pair, token in runs(p, k):
        h, g, u = dH[rows], G[rows], U[rows]
        wr = torch.ones_like(h[:, :1]) if w is None else w.reshape(-1)[pair].double()[:, None]
        top = g.abs().clamp(min=1)
        a = fo.act(name, g)
        t = h * a * u
        dw[0][pair] = t.sum(1)
        dw[1][pair] = (t.shape[1] * EPS * torch.sqrt((t * t).sum(1))
                       + ((h * u).abs() * 2.0 ** -20 * top).sum(1) + SMALL)
        dg, du = wr * h * u * fo.act_grad(name, g), wr * h * a
        eg = (wr * h * u).abs() * 2.0 ** -19 * top
        eu = (wr * h).abs() * 2.0 ** -19 * top
        x1, e1 = fo.rounded_product(dg, Wg[e].t(), eg, True, dtype)
        x2, e2 = fo.rounded_product(du, Wu[e].t(), eu, True, dtype)
        row = x1 + x2
        dX[0].index_add_(0, token, row)
        dX[1].index_add_(0, token, 2 * (e1 + e2))
        size.index_add_(0, token, row.abs())
        for (v, dv), to in ((fo.rounded_product(X[token].t(), dg, eg, False, dtype), dWg),
                            (fo.rounded_product(X[token].t(), du, eu, False, dtype), dWu)):
            to[0][e], to[1][e] = v, fo.stored(v, dv, dtype)
    return dict(dX=(dX[0], fo.stored(dX[0], dX[1] + k * EPS * size, dtype)), dWg=dWg, dWu=dWu,
                dw=tuple(v.view(M, k) for v in dw))
