"""The example that runs the layer operators together: calibration through the
loss's gradient, quantization, and the quantized block's loss."""

import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import torch

    from kronecker_hessian_gptq_gb300 import build as b

    b.build()
    torch.cuda.init()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import quantized_block
    finally:
        sys.path.pop(0)
    return quantized_block


def test_quantization_under_the_calibrated_factors(example):
    """3-bit weights: the solve leaves less of what it minimizes, under the factors of the loss's gradients, than
    rounding to nearest does; and the unquantized block loses the least."""
    out = example.main(tokens=2048, width=256, vocab=4000, bits=3)
    assert out["bakron"][1] < out["rounded"][1], out
    assert out["bf16"][0] < out["bakron"][0], out


def test_eight_bits_keep_the_loss(example):
    """8-bit weights and activations: the loss moves by less than 2% of what 3-bit rounding costs."""
    eight = example.main(tokens=2048, width=256, vocab=4000, bits=8)
    three = example.main(tokens=2048, width=256, vocab=4000, bits=3)
    assert abs(eight["bakron"][0] - eight["bf16"][0]) < 0.02 * (three["rounded"][0] - three["bf16"][0]) + 5e-3, (eight, three)


def test_the_block_in_codes_is_the_block_in_values(example):
    """With codes that stand for the weights exactly, only the activations' codes differ: half a step of each."""
    import torch

    import kronecker_hessian_gptq_gb300 as bk

    block, x, _ = example.make(300, 128, 500)
    codes = torch.randint(-100, 101, (128, 128), device="cuda")
    scales = torch.full((128,), 1 / 1024, device="cuda")
    block["W"] = codes.float() / 1024
    _, n = bk.norm_residual(x, None, pre=block["pre"])
    h = example.run(block, x, codes.to(torch.int8), scales)[3]
    ref = n.double() @ block["W"].double().t()
    step = n.double().abs().amax(1, keepdim=True) / 127
    # the codes come from the norm before it is rounded to bf16, which adds 2^-8 of each of its values
    tol = (0.51 * step * (1 + 2.0 ** -7) + 2.0 ** -8 * n.double().abs()) @ block["W"].double().abs().t() + 2.0 ** -7 * ref.abs() + 1e-6
    assert bool(((h.double() - ref).abs() <= tol).all())
