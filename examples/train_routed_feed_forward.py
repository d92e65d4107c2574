"""Train a routed feed-forward block in 16 bits, then serve it.

One block of a language model, Y = X + the sum over each token's experts of
w (silu(X Wg_e) * (X Wu_e)) Wd_e, is tuned towards a fixed block. A router, logits = X Wr, chooses
k of E experts for every token. Choice and weights come from llmint8_route, the experts' order
of the (token, expert) pairs from llmint8_expert_plan; the plan serves the forward and the
backward products. A bias that only the choice sees is moved towards experts with few tokens
after each step, so that none is left without.

    python examples/train_routed_feed_forward.py [--steps 60] [--tokens 512] [--width 256]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bit_quantized_matmul_col_amd as lm  # noqa: E402

HOW = dict(scores="sigmoid", renormalize=True)


def forward(X, W, k, bias=None, keep=False):
    """Y, and what the backward pass needs when keep is set."""
    Wr, Wg, Wu, Wd = W
    logits = lm.llmint8_matmul(X, Wr)
    ids, weights = lm.llmint8_route(logits, k, bias=bias, **HOW)
    plan = lm.llmint8_expert_plan(ids, Wg.shape[0])
    if not keep:
        H = lm.llmint8_experts_gated(X, Wg, Wu, plan, weights=weights)
        return lm.llmint8_experts_matmul(H, Wd, plan, residual=X), None
    H, G, U = lm.llmint8_experts_gated(X, Wg, Wu, plan, weights=weights, save="full")
    saved = X, logits, ids, weights, plan, H, G, U
    return lm.llmint8_experts_matmul(H, Wd, plan, residual=X), saved


def backward(dY, W, saved):
    """Gradients of the four weights and of X."""
    Wr, Wg, Wu, Wd = W
    X, logits, ids, weights, plan, H, G, U = saved
    dH, dWd = lm.llmint8_experts_matmul_backward(dY, H, Wd, plan)
    dX, dWg, dWu, dweights = lm.llmint8_experts_gated_backward(dH, X, Wg, Wu, G, U, plan,
                                                               weights=weights)
    dlogits = lm.llmint8_route_backward(dweights, logits, ids, **HOW)
    dXr, dWr, _ = lm.llmint8_matmul_backward(dlogits, X, Wr)
    return (dWr, dWg, dWu, dWd), dX + dXr + dY


def setup(width, hidden, experts, dtype, g):
    """(target weights in 16 bits, fp32 weights to train)"""
    shapes = ((width, experts), (experts, width, hidden), (experts, width, hidden),
              (experts, hidden, width))
    target = [torch.randn(s, generator=g, device="cuda") / s[-2] ** 0.5 for s in shapes]
    master = [w + 0.3 * torch.randn(w.shape, generator=g, device="cuda") / w.shape[-2] ** 0.5
              for w in target]
    return [w.to(dtype) for w in target], master


def train(steps=60, tokens=512, width=256, hidden=128, experts=16, k=4, dtype=torch.bfloat16,
          seed=0, lr=2e-3):
    """(losses, weights, bias): Adam on fp32 master weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    target, master = setup(width, hidden, experts, dtype, g)
    first = [torch.zeros_like(w) for w in master]
    second = [torch.zeros_like(w) for w in master]
    bias = torch.zeros(experts, device="cuda")
    losses = []
    for step in range(1, steps + 1):
        X = torch.randn((tokens, width), generator=g, device="cuda").to(dtype)
        want, _ = forward(X, target, k)
        W = [w.to(dtype) for w in master]
        Y, saved = forward(X, W, k, bias, keep=True)
        err = Y.float() - want.float()
        losses.append(err.square().mean())
        grads, _ = backward((err * (2 / tokens)).to(dtype), W, saved)
        for w, a, b, d in zip(master, first, second, grads):
            d = d.float()
            a.mul_(0.9).add_(d, alpha=0.1)
            b.mul_(0.99).addcmul_(d, d, value=0.01)
            w.sub_(lr * (a / (1 - 0.9 ** step)) / ((b / (1 - 0.99 ** step)).sqrt() + 1e-8))
        load = saved[4].offsets.diff().float()
        bias += 1e-3 * torch.sign(tokens * k / experts - load)
    return [float(v) for v in losses], [w.to(dtype) for w in master], bias


def main():
    p = argparse.ArgumentParser()
    for name, value in (("steps", 60), ("tokens", 512), ("width", 256), ("hidden", 128),
                        ("experts", 16), ("k", 4)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    losses, W, bias = train(**vars(a))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    X = torch.randn((1, a.width), device="cuda").to(W[0].dtype)
    print("one token:", forward(X, W, a.k, bias)[0][0, :4].tolist())


if __name__ == "__main__":
    main()
