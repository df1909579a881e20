"""What the Python calls of a projection in 8-bit floats hand to the C entry points, and what they refuse, with
stand-ins for the C entry points and for the tensors' device (no GPU: nothing here is launched)."""

import pytest
import torch

from kronecker_hessian_gptq_gb300 import _layers, _projection
from test_layers_calls_cpu import bf16, entries as _entries_of_layers, f32, on_cuda  # noqa: F401


@pytest.fixture
def entries(_entries_of_layers, monkeypatch):  # noqa: F811
    monkeypatch.setattr(_projection, "_empty", _layers._empty)
    monkeypatch.setattr(_projection, "_entry", _layers._entry)
    return _entries_of_layers


def codes(n, k):
    return on_cuda(torch.zeros((n, k), dtype=torch.uint8))


def states(*sizes):
    return {k: [f32(n) for n in sizes] for k in "mv"}


@pytest.mark.parametrize("name,call", [
    ("bakron_fp8_matmul", lambda: _projection.fp8_matmul(bf16(40, 256), codes(130, 256), f32(2, 2))),
    ("bakron_fp8_matmul_backward", lambda: _projection.fp8_matmul_backward(bf16(40, 130), bf16(40, 256), codes(130, 256), f32(2, 2))),
    ("bakron_head_norm_rotary_backward",
     lambda: _projection.head_norm_rotary_backward(bf16(6, 4, 64), None, bf16(6, 4, 64), None, None, None, f32(64))),
    ("bakron_adamw", lambda: _projection.adamw([f32(9), f32(3, 4)], [bf16(9), f32(12)], states(9, 12), 1)),
])
def test_the_workspace_lives_until_the_call_has_returned(entries, name, call):
    """Memory that is given back before the launches can be handed to another thread, or unmapped, meanwhile."""
    call()
    assert entries == [(name, True)]


@pytest.mark.parametrize("call", [
    lambda: _projection.quantize_blocks(bf16(4, 64), (64, 64)),
    lambda: _projection.quantize_blocks(bf16(4, 64)[:, ::2]),
    lambda: _projection.fp8_matmul(bf16(4, 64), codes(8, 65), f32(1, 1)),
    lambda: _projection.fp8_matmul(bf16(4, 64), codes(8, 64), f32(1, 2)),
    lambda: _projection.fp8_matmul(bf16(4, 64), codes(8, 64), None),
    lambda: _projection.fp8_matmul(bf16(4, 64), codes(8, 64), f32(1, 1), bias=f32(7)),
    lambda: _projection.fp8_matmul(bf16(1, 64).expand(4, 64), codes(8, 64), f32(1, 1)),
    lambda: _projection.fp8_matmul_backward(bf16(4, 8), bf16(5, 64), codes(8, 64), f32(1, 1)),
    lambda: _projection.fp8_matmul_backward(bf16(4, 9), bf16(4, 64), codes(8, 64), f32(1, 1)),
    lambda: _projection.head_norm_rotary(bf16(4, 2, 64), bf16(3, 1, 64), None, None),
    lambda: _projection.head_norm_rotary(bf16(4, 2, 64), None, None, on_cuda(torch.ones(4, dtype=torch.float64))),
    lambda: _projection.head_norm_rotary(bf16(4, 2, 64)[..., ::2], None, None, None),
    lambda: _projection.adamw([f32(9)], [bf16(8)], states(9), 1),
    lambda: _projection.adamw([f32(9)], [bf16(9)], states(8), 1),
    lambda: _projection.adamw([f32(4, 4).t()], [bf16(16)], states(16), 1),
    lambda: _projection.adamw([f32(9)], [on_cuda(torch.zeros(9, dtype=torch.float64))], states(9), 1),
    lambda: _projection.adamw([f32(9), f32(3)], [f32(9), f32(3)], states(9), 1),
    lambda: _projection.adamw([f32(9)], [f32(9)], states(9), 1, copies=[f32(9)]),
])
def test_refusals(entries, call):
    with pytest.raises(ValueError):
        call()
    assert not entries
