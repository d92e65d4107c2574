"""Train a gated feed-forward block in 16 bits, then serve it.

One block of a language model, Y = X + (silu(X Wg) * (X Wu)) Wd, is tuned towards a fixed
block whose weights differ from its own by 30 %. What the backward pass needs is kept as 8-bit checkpoints:
X (llmint8_checkpoint_pack), the pre-activations (from the gated kernel's epilogue) and H.
The weights stay [K, N] throughout, so after training they go to llmint8_quantize_colwise
unchanged, and a single token runs through the 16-bit block and through its int8 layers.

    python examples/train_feed_forward.py [--steps 60] [--tokens 512] [--width 256] [--hidden 704]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bit_quantized_matmul_col_amd as lm  # noqa: E402


def forward(X, W, keep):
    """Y, and what the backward pass needs when keep is set."""
    Wg, Wu, Wd = W
    if not keep:
        H = lm.llmint8_gated(X, Wg, Wu)
        return lm.llmint8_matmul(H, Wd, residual=X), None
    H, G, U = lm.llmint8_gated(X, Wg, Wu, save="8bit")
    saved = (lm.llmint8_checkpoint_pack(X), G, U, lm.llmint8_checkpoint_pack(H))
    return lm.llmint8_matmul(H, Wd, residual=X), saved


def backward(dY, W, saved):
    """Gradients of the three weights and of X."""
    Wg, Wu, Wd = W
    X, G, U, H = saved
    dH, dWd, _ = lm.llmint8_matmul_backward(dY, H, Wd)
    dX, dWg, dWu = lm.llmint8_gated_backward(dH, X, Wg, Wu, G, U)
    return (dWg, dWu, dWd), dX + dY


def setup(width, hidden, dtype, g):
    """(target weights in 16 bits, fp32 weights to train)"""
    shapes = ((width, hidden), (width, hidden), (hidden, width))
    target = [torch.randn(s, generator=g, device="cuda") / s[0] ** 0.5 for s in shapes]
    master = [w + 0.3 * torch.randn(w.shape, generator=g, device="cuda") / w.shape[0] ** 0.5
              for w in target]
    return [w.to(dtype) for w in target], master


def train(steps=60, tokens=512, width=256, hidden=704, dtype=torch.bfloat16, seed=0, lr=2e-3):
    """(losses, weights): Adam on fp32 master weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    target, master = setup(width, hidden, dtype, g)
    first = [torch.zeros_like(w) for w in master]
    second = [torch.zeros_like(w) for w in master]
    losses = []
    for step in range(1, steps + 1):
        X = torch.randn((tokens, width), generator=g, device="cuda").to(dtype)
        want, _ = forward(X, target, keep=False)
        W = [w.to(dtype) for w in master]
        Y, saved = forward(X, W, keep=True)
        err = Y.float() - want.float()
        losses.append(err.square().mean())
        grads, _ = backward((err * (2 / tokens)).to(dtype), W, saved)
        for w, a, b, d in zip(master, first, second, grads):
            d = d.float()
            a.mul_(0.9).add_(d, alpha=0.1)
            b.mul_(0.99).addcmul_(d, d, value=0.01)
            w.sub_(lr * (a / (1 - 0.9 ** step)) / ((b / (1 - 0.99 ** step)).sqrt() + 1e-8))
    return [float(v) for v in losses], [w.to(dtype) for w in master]


def serve_int8(X, W):
    """The block with its three products as LLM.int8() layers (fp16)."""
    Wg, Wu, Wd = (w.half() for w in W)
    quant = [(w, *lm.llmint8_quantize_colwise(w)) for w in (Wg, Wu, Wd)]

    def linear(x, layer):
        w, codes, absmax = layer
        return lm.llmint8_linear(x, codes, absmax, w)
    H = (torch.nn.functional.silu(linear(X, quant[0]).float())
         * linear(X, quant[1]).float()).half()
    return X + linear(H, quant[2])


def main():
    p = argparse.ArgumentParser()
    for name, value in (("steps", 60), ("tokens", 512), ("width", 256), ("hidden", 704)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    losses, W = train(a.steps, a.tokens, a.width, a.hidden)
    for i in range(0, len(losses), max(1, len(losses) // 6)):
        print(f"step {i + 1:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses):4d}  loss {losses[-1]:.4f}")
    X = torch.randn((1, a.width), generator=torch.Generator(device="cuda").manual_seed(9),
                    device="cuda").half()
    half = [w.half() for w in W]
    y16, _ = forward(X, half, keep=False)
    y8 = serve_int8(X, half)
    off = float((y8.float() - y16.float()).norm() / y16.float().norm())
    print(f"one token: int8 layers against the 16-bit block, relative difference {off:.4f}")


if __name__ == "__main__":
    main()
