"""An AdamW step changes leaves of autograd in place, and autograd knows it: a graph made before the step that kept a
parameter refuses to go backward with the new values, as it does after a step of torch's own optimizers."""

import pytest

from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_graph_from_before_the_step(bk, bits, native, monkeypatch):  # noqa: F811
    import torch

    from kronecker_hessian_gptq_gb300 import _projection

    if not native:  # the call through ctypes
        class Nothing:
            @staticmethod
            def adamw(*args):
                return None

        monkeypatch.setattr(_projection, "_native", Nothing)
    w = [torch.randn(300, device="cuda", requires_grad=True), torch.randn((3, 5), device="cuda", requires_grad=True)]
    copies = [torch.zeros(300, dtype=torch.bfloat16, device="cuda"), None]
    states = bk.adamw_states(w, bits)
    seen = lambda: [t._version for l in (w, copies[:1]) for t in l]  # noqa: E731
    loss = sum((p * p).sum() for p in w)
    kept = (copies[0].detach().requires_grad_() * copies[0]).sum()
    grads = list(torch.autograd.grad(loss, w, retain_graph=True))
    versions, old = seen(), [g._version for g in grads]
    bk.adamw(w, grads, states, 1, copies=copies)
    assert all(a > b for a, b in zip(seen(), versions)) and [g._version for g in grads] == old
    for stale in (loss, kept):
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            stale.backward()
    # a graph of the new values goes
    new = torch.autograd.grad(sum((p * p).sum() for p in w), w)
    assert all(torch.equal(g, 2 * p.detach()) for g, p in zip(new, w))


def test_tensors_without_a_version(bk):  # noqa: F811
    import torch

    with torch.inference_mode():
        p = [torch.zeros(300, device="cuda")]
        g, states = [torch.ones(300, device="cuda")], bk.adamw_states(p)
        assert int(bk.adamw(p, g, states, 1).item()) == 0
    assert int(bk.adamw(p, g, states, 2).item()) == 0 and bool((p[0] < 0).all())


def test_a_refused_step_changes_no_version(bk):  # noqa: F811
    import torch

    p = [torch.zeros(300, device="cuda")]
    states = bk.adamw_states(p)
    with pytest.raises(RuntimeError):
        bk.adamw(p, p, states, 1)
    assert p[0]._version == 0
