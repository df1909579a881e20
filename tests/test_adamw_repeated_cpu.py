"""bakron_adamw refuses a list in which anything that a step writes is there twice, whatever its two places: two blocks
would write it at once.  (No GPU: a refused call launches nothing, and none here is accepted.)"""

import ctypes
import itertools

import pytest

from test_layers_abi_cpu import BF16, F32, at, lib  # noqa: F401
from test_projection_abi_cpu import Tensor

WRITTEN = ["param", "m", "v", "ms", "vs", "copy"]


def _step(lib, tensors, bits=8):  # noqa: F811
    array = (Tensor * len(tensors))(*tensors)
    return lib.bakron_adamw(array, len(tensors), bits, 1e-3, None, 1, None, 0.9, 0.99, 1e-8, 0.1, 1.0, None, None, 0, None, 0,
                            at(0x8000), None)


def _tensors(n=3):
    out = []
    for i in range(n):
        base = 0x100000 * (i + 1)
        out.append(dict(param=base, grad=base + 0x1000, m=base + 0x2000, v=base + 0x3000, ms=base + 0x4000, vs=base + 0x5000,
                        copy=base + 0x6000, n=9, pt=F32, gt=BF16, ct=BF16))
    return out


INVALID, WORKSPACE = 1, 4  # without a workspace a list that is in order is refused for that, after it was looked at


def test_different_tensors(lib):  # noqa: F811
    assert _step(lib, [Tensor(**t) for t in _tensors(200)]) == WORKSPACE


@pytest.mark.parametrize("first,second", list(itertools.product(WRITTEN, WRITTEN)))
def test_the_same_array_in_two_tensors(lib, first, second):  # noqa: F811
    t = _tensors()
    t[2][second] = t[0][first]
    assert _step(lib, [Tensor(**x) for x in t]) == INVALID


@pytest.mark.parametrize("first,second", list(itertools.combinations(WRITTEN, 2)))
def test_the_same_array_twice_in_a_tensor(lib, first, second):  # noqa: F811
    t = _tensors()
    t[1][second] = t[1][first]
    assert _step(lib, [Tensor(**x) for x in t]) == INVALID


def test_scales_do_not_count_with_32_bits_nor_do_empty_tensors(lib):  # noqa: F811
    t = _tensors()
    t[1]["ms"] = t[0]["ms"]
    assert _step(lib, [Tensor(**x) for x in t], 32) == WORKSPACE
    t[1].update({k: t[0][k] for k in WRITTEN}, n=0)
    assert _step(lib, [Tensor(**x) for x in t]) == WORKSPACE
    for x in t:  # a gradient may be that of several
        x["grad"] = t[0]["grad"]
    assert _step(lib, [Tensor(**x) for x in t]) == WORKSPACE
