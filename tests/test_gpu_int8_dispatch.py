"""The 8-bit product on both sides of every choice it makes by size: each form of the row kernel, warps with several rows,
tiles in turns, shares of K that run from one tile into the next, prompts of several tiles for each pair of SMs.  Against
exact sums, with the tolerances of test_gpu_int8_matmul.py."""

import numpy as np
import pytest

from test_gpu_int8_matmul import U, _reference_codes, bk  # noqa: F401

pytestmark = pytest.mark.gpu


def _inputs(t, k, n, seed):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((t, k), generator=gen, device="cuda") * (1 + 7 * (torch.rand(k, generator=gen, device="cuda") < 0.05))
    v = torch.randint(-128, 128, (n, k), generator=gen, device="cuda", dtype=torch.int16).to(torch.int8)
    w = 1e-4 + 9e-4 * torch.rand(n, generator=gen, device="cuda")
    b = torch.randn(n, generator=gen, device="cuda")
    return x, v, w, b


def _check(y, c, s, v, w, b, dtype):
    """Against the codes' exact sums (fp64 products of 8-bit codes: below 2^53), scaled in fp64."""
    main = (c.double() @ v.double().t()) * s.double()[:, None] * w.double()
    ref = main if b is None else main + b.double()
    tol = (4 * main.abs() + ref.abs()) * 2.0 ** -24 + U[dtype] * ref.abs() * (1 + 2.0 ** -8) + (2.0 ** -25 if dtype == "float16" else 0)
    assert y.shape == ref.shape
    worst = float(((y.double() - ref).abs() / tol.clamp(min=1e-300)).max())
    assert worst <= 1.0, worst


def _all_forms(bk, t, k, n, types=("float32", "bfloat16")):  # noqa: F811
    import torch

    x, v, w, b = _inputs(t, k, n, t + k + n)
    for dtype in types:
        xt = x.to(getattr(torch, dtype))
        c, s = _reference_codes(xt)
        c, s = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
        y, st = bk.int8_matmul(xt, v, w, bias=b)
        assert int(st.item()) == 0
        _check(y, c, s, v, w, b, dtype)
        y, st = bk.int8_matmul(c, v, w, x_scales=s, dtype=xt.dtype)
        assert int(st.item()) == 0
        _check(y, c, s, v, w, None, dtype)


@pytest.mark.parametrize("t", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("k,n", [(4096, 300), (4099, 300), (4096, 14336), (4099, 14336), (512, 9731), (16, 5000)])
def test_a_few_tokens(bk, t, k, n):  # noqa: F811
    """By rows up to four tokens: a row shared by warps, one for each warp, several one after another (more than 4864)."""
    _all_forms(bk, t, k, n)


@pytest.mark.parametrize("t,k,n", [
    (512, 1024, 8192),   # 128 whole tiles for 76 pairs: a second tile with its sums in the same tensor memory
    (700, 640, 8200),    # 198 tiles, 117 tokens each
    (128, 2049, 20000),  # 79 tiles: equal shares of K run from one tile into the next
    (129, 14336, 4096),  # 32 tiles of 96 tokens, two pairs for each
    (256, 8192, 9900),   # 78 tiles of 64 steps: a last wave of two
    (128, 5000, 300), (129, 5000, 300), (64, 3000, 5000), (65, 3000, 5000), (96, 1024, 12288), (160, 1100, 10000),
    (768, 1040, 1000), (767, 4099, 515)])
def test_batches(bk, t, k, n):  # noqa: F811
    _all_forms(bk, t, k, n, ("float32", "float16"))


@pytest.mark.parametrize("t,k,n", [(769, 300, 9000), (1100, 512, 14336), (1025, 2050, 5000), (2049, 1100, 4100)])
def test_prompts(bk, t, k, n):  # noqa: F811
    """Several tiles for each pair of SMs, with rows of results on 16 bytes and not, sums of one and of three segments."""
    _all_forms(bk, t, k, n, ("float32", "bfloat16"))
