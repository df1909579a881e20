"""The product of e4m3 codes and its gradients with more rows than one group of tiles has (4096), where a pair of SMs
goes on to another tile after one at the matrix's right edge.  Widths of every kind of edge: tiles have 256 columns,
of which a warp holds 64 and, 128 further on, 64 more, and either may lie outside.  Bounds as in
test_gpu_fp8_matmul.py; and the same call gives the same results bit for bit."""

import numpy as np
import pytest

from test_gpu_fp8_matmul import _check, _layer, _numbers, _quantized
from test_gpu_int8_matmul import _values, bk  # noqa: F401

pytestmark = pytest.mark.gpu

EDGES = [8, 64, 104, 128, 136, 168, 192, 200]


def _repeats(call, want, times=8):
    import torch

    for _ in range(times):
        assert torch.equal(call(), want)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("k", [64, 128, 1408])
@pytest.mark.parametrize("edge", EDGES)
def test_product(bk, edge, k, dtype):  # noqa: F811
    rng = np.random.default_rng(edge + k)
    t, n = 16384 + 5, 512 + edge
    x, (v, w) = _values(rng, t, k, dtype), _layer(bk, rng, n, k)
    y, st = bk.fp8_matmul(x, v, w)
    assert int(st.item()) == 0
    c, s = _quantized(x, 1, 128)
    _check(y, _numbers(c.cuda(), s.cuda(), 1, 128), _numbers(v, w, 128, 128), -(-k // 128))
    _repeats(lambda: bk.fp8_matmul(x, v, w)[0], y)


@pytest.mark.parametrize("t,n", [(8192, 1408), (30000, 896), (16384, 1664)])
def test_product_with_a_bias_and_given_codes(bk, t, n):  # noqa: F811
    import torch

    rng = np.random.default_rng(t + n)
    x, (v, w) = _values(rng, t, 192, "bfloat16"), _layer(bk, rng, n, 192)
    bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
    y, st = bk.fp8_matmul(x, v, w, bias=bias)
    assert int(st.item()) == 0
    c, s = bk.quantize_blocks(x)
    _check(y, _numbers(c, s, 1, 128), _numbers(v, w, 128, 128), 2, bias)
    assert torch.equal(bk.fp8_matmul(c, v, w, x_scales=s, bias=bias, dtype=torch.bfloat16)[0], y)
    _repeats(lambda: bk.fp8_matmul(x, v, w, bias=bias)[0], y)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("n", [64, 128, 1408])
@pytest.mark.parametrize("edge", EDGES)
def test_gradient_of_the_values(bk, edge, n, dtype):  # noqa: F811
    rng = np.random.default_rng(edge + n)
    t, k = 16384 + 5, 512 + edge
    dy, (v, w) = _values(rng, t, n, dtype), _layer(bk, rng, n, k)
    g, st = bk.fp8_matmul_backward(dy, None, v, w)
    assert int(st.item()) == 0
    c, s = _quantized(dy, 1, 128)
    _check(g["X"], _numbers(c.cuda(), s.cuda(), 1, 128), _numbers(v, w, 128, 128).t(), -(-n // 128))
    _repeats(lambda: bk.fp8_matmul_backward(dy, None, v, w)[0]["X"], g["X"])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("t", [64, 128, 1408])
@pytest.mark.parametrize("edge", EDGES)
def test_gradient_of_the_weights(bk, edge, t, dtype):  # noqa: F811
    import torch

    rng = np.random.default_rng(edge + t)
    n, k = 16384 + 8, 512 + edge
    dy, x, (v, w) = _values(rng, t, n, dtype), _values(rng, t, k, dtype), _layer(bk, rng, n, k)
    g, st = bk.fp8_matmul_backward(dy, x, v, w)
    assert int(st.item()) == 0

    def of(m):
        c, s = _quantized(m, 128, 1)
        return _numbers(c.cuda(), s.cuda(), 128, 1)

    # A block of tokens has a scale for each row and each column: one rounding more
    _check(g["W"], of(dy).t(), of(x).t(), -(-t // 128) + 1)
    for _ in range(8):
        again = bk.fp8_matmul_backward(dy, x, v, w)[0]
        assert torch.equal(again["W"], g["W"]) and torch.equal(again["X"], g["X"])
