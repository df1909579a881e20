"""A step's parameters and copies count as changed in place, its gradients do not (stand-ins as in
test_projection_calls_cpu.py; no GPU)."""

import pytest

from kronecker_hessian_gptq_gb300 import _projection
from test_layers_calls_cpu import bf16, entries as _entries_of_layers, f32, on_cuda  # noqa: F401
from test_projection_calls_cpu import entries  # noqa: F401


@pytest.mark.parametrize("bits", [8, 32])
def test_autograd_sees_what_a_step_changes(entries, bits):  # noqa: F811
    p, g = [f32(300), f32(3, 4)], [bf16(300), f32(12)]
    state = {k: [on_cuda(t) for t in l] for k, l in _projection.adamw_states(p, bits).items()}
    copies = [bf16(300), None]
    _projection.adamw(p, g, state, 1, copies=copies)
    assert all(t._version == 1 for l in (p, copies[:1]) for t in l) and all(t._version == 0 for t in g)
    with pytest.raises(ValueError):
        _projection.adamw(p, g[:1], state, 1)
    assert all(t._version == 1 for t in p)
