"""What the layer operators' Python calls hand to the C entry points, with stand-ins for the C
entry points and for the tensors' device (no GPU: nothing here is launched)."""

import weakref

import pytest
import torch

from kronecker_hessian_gptq_gb300 import _layers


class OnCuda(torch.Tensor):
    """A CPU tensor that says it is on cuda:0; the calls only read its address."""

    is_cuda = True

    def get_device(self):
        return 0


def on_cuda(t):
    return torch.Tensor._make_subclass(OnCuda, t)


def bf16(*shape):
    return on_cuda(torch.zeros(shape, dtype=torch.bfloat16))


def f32(*shape):
    return on_cuda(torch.zeros(shape))


@pytest.fixture
def entries(monkeypatch):
    """Stands in for the C library: every workspace size is `size`; a call checks that memory of that size, of a tensor
    that still lives, is among its arguments."""
    size, made, calls = 4096, [], []

    def empty(*args, **kw):
        t = torch.empty(*args, **kw)
        made.append((weakref.ref(t), t.data_ptr(), t.numel() * t.element_size()))
        return t

    def entry(name):
        if name.endswith("workspace_size"):
            return lambda *args: size

        def call(*args):
            at = args.index(size)
            alive = [p for ref, p, n in made if ref() is not None and n == size]
            calls.append((name, args[at - 1] in alive))
            return 0

        return call

    monkeypatch.setattr(_layers, "_empty", empty)
    monkeypatch.setattr(_layers, "_entry", entry)
    monkeypatch.setattr(_layers, "_current_device", lambda: 0)
    monkeypatch.setattr(_layers, "_handle", lambda device: 0)
    return calls


@pytest.mark.parametrize("name,call", [
    ("bakron_int8_matmul",
     lambda: _layers.int8_matmul(bf16(40, 64), on_cuda(torch.zeros((16, 64), dtype=torch.int8)), f32(16))),
    ("bakron_norm_residual_backward",
     lambda: _layers.norm_residual_backward(bf16(6, 64), None, bf16(6, 64), bf16(6, 64), post=f32(64))),
    ("bakron_linear_cross_entropy",
     lambda: _layers.linear_cross_entropy(bf16(6, 64), bf16(9, 64), on_cuda(torch.zeros(6, dtype=torch.int64)))),
    ("bakron_linear_cross_entropy_grad",
     lambda: _layers.linear_cross_entropy_grad(bf16(6, 64), bf16(9, 64), on_cuda(torch.zeros(6, dtype=torch.int64)))),
])
def test_the_workspace_lives_until_the_call_has_returned(entries, name, call):
    """Memory that is given back before the launches can be handed to another thread, or unmapped, meanwhile."""
    call()
    assert entries == [(name, True)]


def test_a_library_without_an_entry_point_is_named(monkeypatch):
    """An older libbakron.so than the package's own: the error says which file and what it lacks."""
    from kronecker_hessian_gptq_gb300 import _lib
    from kronecker_hessian_gptq_gb300 import build as b

    b.build()
    monkeypatch.setattr(_lib, "_lib", None)
    monkeypatch.setitem(_lib.SIGNATURES, "bakron_of_a_later_version", (None, []))
    with pytest.raises(RuntimeError, match="libbakron.so.*bakron_of_a_later_version.*build it again"):
        _lib.load()
