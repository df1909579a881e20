"""One residual block of a language model, from calibration to its quantized run.

    h = W N(x),  y = x + gate * N(h),  loss = cross entropy of N(y) under the head

  1. calibration   the loss's gradient with respect to N(y), taken back through the
                   norms to the layer's output h; the Grams of the layer's inputs and
                   of these gradients are the Kronecker factors A and B
  2. quantization  BaKron of W under A (x) B, and plain rounding for comparison
  3. the run       (on other tokens) the norm's output as 8-bit codes into the 8-bit product, the block's
                   end and the next norm in one call, and the loss of the result

    python examples/quantized_block.py [--tokens 4096 --width 1024 --vocab 32768 --bits 3]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import kronecker_hessian_gptq_gb300 as bk  # noqa: E402

BF16 = torch.bfloat16


def make(tokens, width, vocab, seed=0):
    """Random weights, and hidden states with a few loud features and targets that the head partly knows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    loud = 1 + 5 * (torch.rand(width, generator=gen, device="cuda") < 0.02)
    # features that share a few directions, as a layer's inputs do
    few = max(4, width // 16)
    mix = rand(few, width) * few ** -0.5
    block = {"W": rand(width, width) * width ** -0.5, "pre": 1 + 0.1 * rand(width), "post": 1 + 0.1 * rand(width),
             "next": 1 + 0.1 * rand(width), "gate": (1 + 0.2 * rand(width)).to(BF16),
             "head": (rand(vocab, width) * 4 * width ** -0.5).to(BF16)}
    x = ((rand(tokens, few) @ mix + 0.2 * rand(tokens, width)) * loud).to(BF16)
    z = run(block, x)[1]  # what the block itself would predict, with some noise
    scores = z.float() @ block["head"].float().t() + 2 * rand(tokens, vocab)
    return block, x, scores.argmax(1)


def run(block, x, codes=None, scales=None):
    """The block in bf16, or with its layer in 8-bit codes: (y, N(y), N(x), h)."""
    n = None
    if codes is None:
        _, n = bk.norm_residual(x, None, pre=block["pre"])
        h = n @ block["W"].to(BF16).t()
    else:
        _, c, s = bk.norm_residual(x, None, pre=block["pre"], codes=True)
        h, status = bk.int8_matmul(c, codes, scales, x_scales=s, dtype=BF16)
        assert int(status.item()) == 0
    y, z = bk.norm_residual(x, h, post=block["post"], gate=block["gate"], pre=block["next"])
    return y, z, n, h


def mean_loss(block, z, targets):
    loss, _, status = bk.linear_cross_entropy(z, block["head"], targets)
    assert int(status.item()) == 0
    return float(loss.mean())


def factors(block, x, targets):
    """A and B of the layer: Grams of its inputs and of the loss's gradients at its outputs."""
    y, z, n, h = run(block, x)
    each = torch.ones(len(x), device="cuda")  # one gradient for each token, not for the mean
    _, _, dz, _, status = bk.linear_cross_entropy_grad(z, block["head"], targets, coef=each)
    assert int(status.item()) == 0
    grads = bk.norm_residual_backward(None, dz, y, h, post=block["post"], gate=block["gate"], pre=block["next"])
    A, _ = bk.gram(n.t().contiguous())
    B, _ = bk.gram(grads["H"].t().contiguous())
    return bk.damp(A, 0.01), bk.damp(B, 0.01)


def main(tokens=4096, width=1024, vocab=32768, bits=3, seed=0):
    block, x, targets = make(tokens, width, vocab, seed)
    half = tokens // 2  # calibrate on one half, judge on the other
    A, B = factors(block, x[:half], targets[:half])
    LA, LB, info = bk.prepare(A, B)
    lo, hi = -(1 << (bits - 1)), (1 << (bits - 1)) - 1
    scales = bk.row_scales(block["W"], lo, hi, grid=20)
    V, Wq, status = bk.quantize_range(block["W"], LA, LB, scales, lo, hi)
    assert int(status.item()) == 0 and not info.any()
    rounded = torch.clamp(torch.round(block["W"] / scales[:, None]), lo, hi)
    x, targets = x[half:], targets[half:]
    out = {"bf16": (mean_loss(block, run(block, x)[1], targets), 0.0)}
    for name, codes in (("rounded", rounded), ("bakron", V)):
        E = codes * scales[:, None] - block["W"]  # what is minimized: tr(B E A E^T)
        out[name] = (mean_loss(block, run(block, x, codes.to(torch.int8), scales)[1], targets), float(((B @ E @ A) * E).sum()))
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("width", 1024), ("vocab", 32768), ("bits", 3), ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    for name, (loss, distortion) in main(**vars(ap.parse_args())).items():
        print(f"{name:8s} mean loss {loss:.4f}  distortion {distortion:.4g}")
