"""One token expanded over all positions (a stride of 0 between tokens), whose heads lie side by side, have a gap between
them, or lie off 16 bytes: the results of the same tokens written out, within twice the bound of test_gpu_head_norm.py
where another variant may sum a head's squares in another order, and their gradients likewise."""

import numpy as np
import pytest

from test_gpu_head_norm import E, _args, _inputs, _normed, _own, _turned
from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("pad", [0, 1, 4, 8])
@pytest.mark.parametrize("t,h,d", [(40, 4, 64), (2, 3, 128), (6, 5, 48), (1500, 2, 77)])
def test_an_expanded_token(bk, t, h, d, pad, pairs, dtype):  # noqa: F811
    import torch

    rng = np.random.default_rng(t + d + pad)
    p, f, (w, _) = _args(rng, t, d, d // 2 // 16 * 16 + 16, start=5)
    q, _ = _inputs(rng, 1, h, 1, d, dtype, pad=pad)
    one = q.expand(t, h, d)
    whole = one.contiguous()
    got = bk.head_norm_rotary(one, None, p, f, w, None, 1e-6, pairs)[0]
    want, size = _turned(_normed(whole, w, 1e-6), p, f, pairs)
    u, least = _own(dtype)
    assert bool(((got.double() - want).abs() <= 32 * E * size + u * want.abs() + least).all())
    # and as the result's gradient, which every position turns back by its own angle
    x, _ = _inputs(rng, t, h, 1, d, dtype)
    a = bk.head_norm_rotary_backward(one, None, x, None, p, f, w, None, 1e-6, pairs)
    b = bk.head_norm_rotary_backward(whole, None, x, None, p, f, w, None, 1e-6, pairs)
    r = (x.double().pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
    dn, both = _turned(whole.double(), p, f, pairs, back=True)
    unit, g = x.double() * r, both * w.double().abs()
    terms = (g + unit.abs() * (g * unit.abs()).mean(-1, keepdim=True)) * r
    assert bool(((a["Q"].double() - b["Q"].double()).abs() <= 128 * E * terms + 2 * u * b["Q"].double().abs() + 2 * least).all())
    # sums of blocks' sums, in a tree at most 128 deep either way
    assert bool(((a["q_weight"].double() - b["q_weight"].double()).abs() <= 2 * 192 * E * (both * unit.abs()).sum((0, 1))).all())
