"""A projection of queries and keys, quantized by the solve and trained on in 8-bit floats.

    y = x V^T,   (q, k) = rotary(N(y)),   loss = mean (q - q*)^2 + mean (k - k*)^2

  1. the teacher    the projection in bf16, its heads' norms and the rotation
  2. the start      the solve's codes of W under the Gram of the inputs (3 bits)
  3. a step         V = W in e4m3 blocks of 128, the product, the heads, the loss's
                    gradient back through both, AdamW on W and on the norms' weights
                    with states in 8 bits

    python examples/trained_projection.py [--tokens 4096 --width 1024 --steps 50]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import kronecker_hessian_gptq_gb300 as bk  # noqa: E402

BF16 = torch.bfloat16


def make(tokens, width, queries, keys, head, bits, seed=0):
    """Inputs with a few loud features, the teacher's results, and the parameters that training starts from."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    loud = 1 + 5 * (torch.rand(width, generator=gen, device="cuda") < 0.02)
    few = max(4, width // 16)
    x = ((rand(tokens, few) @ (rand(few, width) * few ** -0.5) + 0.2 * rand(tokens, width)) * loud).to(BF16)
    W = rand((queries + keys) * head, width) * width ** -0.5
    layer = {"queries": queries, "keys": keys, "head": head, "positions": torch.arange(tokens, device="cuda"),
             "freqs": 10000.0 ** (-torch.arange(0, head, 2, dtype=torch.float64, device="cuda") / head)}
    params = {"W": W, "q": 1 + 0.2 * rand(head), "k": 1 + 0.2 * rand(head)}
    target = heads(layer, params, x @ W.to(BF16).t())
    A, _ = bk.gram(x[: tokens // 8 * 8].t().contiguous())
    LA, _, info = bk.prepare(bk.damp(A, 0.01), torch.eye(len(W), device="cuda"))
    assert not info.any()
    lo, hi = -(1 << (bits - 1)), (1 << (bits - 1)) - 1
    _, start, status = bk.quantize_range(W, LA, None, bk.row_scales(W, lo, hi, grid=20), lo, hi)
    assert int(status.item()) == 0
    return layer, x, target, {**params, "W": start}


def heads(layer, params, y):
    """Queries and keys of the projection's output y."""
    y = y.view(len(y), layer["queries"] + layer["keys"], layer["head"])
    return bk.head_norm_rotary(y[:, : layer["queries"]], y[:, layer["queries"] :], layer["positions"], layer["freqs"],
                               q_weight=params["q"], k_weight=params["k"])


def gradients(layer, params, x, target):
    """The loss and its gradients in W and the norms' weights; W taken in e4m3 blocks."""
    V, scales = bk.quantize_blocks(params["W"], (128, 128))
    y, status = bk.fp8_matmul(x, V, scales)
    out = heads(layer, params, y)
    off = [a.float() - b.float() for a, b in zip(out, target)]
    loss = sum((e * e).mean() for e in off)
    dq, dk = ((e * (2 / e.numel())).to(BF16) for e in off)
    y = y.view(len(y), layer["queries"] + layer["keys"], layer["head"])
    back = bk.head_norm_rotary_backward(dq, dk, y[:, : layer["queries"]], y[:, layer["queries"] :], layer["positions"],
                                        layer["freqs"], q_weight=params["q"], k_weight=params["k"])
    dy = torch.cat([back["Q"], back["K"]], 1).view(len(x), -1)
    grads, status2 = bk.fp8_matmul_backward(dy, x, V, scales)
    return loss, {"W": grads["W"], "q": back["q_weight"], "k": back["k_weight"]}, status | status2


def main(tokens=4096, width=1024, queries=8, keys=2, head=128, bits=3, steps=50, lr=2e-4, seed=0):
    layer, x, target, params = make(tokens, width, queries, keys, head, bits, seed)
    names = list(params)
    states = bk.adamw_states([params[n] for n in names], bits=8)
    losses = []
    for step in range(1, steps + 1):
        loss, grads, status = gradients(layer, params, x, target)
        losses.append(loss)
        status |= bk.adamw([params[n] for n in names], [grads[n] for n in names], states, step, lr=lr, betas=(0.9, 0.95),
                           weight_decay=0.0, seed=seed)
        assert int(status.item()) == 0
    return [float(v) for v in losses], params


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("width", 1024), ("queries", 8), ("keys", 2), ("head", 128), ("bits", 3), ("steps", 50),
                        ("seed", 0)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--lr", type=float, default=2e-4)
    history, _ = main(**vars(ap.parse_args()))
    for i in sorted({0, *range(9, len(history), 10), len(history) - 1}):
        print(f"step {i + 1:4d}  loss {history[i]:.5f}")
