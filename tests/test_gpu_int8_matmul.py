"""8-bit codes of activations (bakron_quantize_tokens) and the product of
quantized activations and weights (bakron_int8_matmul).

Codes and scales are defined by single fp32 operations (a division, a
division, a rounding to an integer), so they must be equal.  In the product
the sum over k is exact in integers; what is rounded is its conversion to
fp32, the two scalings and the bias: at most four roundings of 2^-24 of
|s w sum|, one of the result, and the output type's own, u (2^-24, 2^-11,
2^-8 for fp32, fp16, bf16; fp16 adds half its smallest step, 2^-25)."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


@pytest.fixture(scope="module")
def bk():
    import torch

    import kronecker_hessian_gptq_gb300 as bk
    from kronecker_hessian_gptq_gb300 import build as b

    b.build()
    bk.load_library()
    torch.cuda.init()
    return bk


def _codes(rng, n, k):
    import torch

    return torch.from_numpy(rng.integers(-128, 128, size=(n, k)).astype(np.int8)).cuda()


def _values(rng, t, k, dtype):
    import torch

    x = rng.standard_normal((t, k)) * np.where(rng.random(k) < 0.05, 8.0, 1.0)
    return torch.from_numpy(x.astype(np.float32)).cuda().to(getattr(torch, dtype))


def _reference_codes(x):
    """The definition in fp32, on the host (IEEE division, rint to even)."""
    x = x.float().cpu().numpy()
    s = (np.abs(x).max(axis=1) / np.float32(127)).astype(np.float32)
    q = x / np.where(s > 0, s, np.float32(1))[:, None]
    assert q.dtype == np.float32
    return np.clip(np.rint(q), -127, 127).astype(np.int8), s


def _check(Y, c, s, v, w, bias, dtype):
    """Against exact integer sums of the codes, scaled in fp64."""
    total = c.astype(np.float64) @ v.astype(np.float64).T  # below 2^53: exact
    main = total * s.astype(np.float64)[:, None] * w.astype(np.float64)
    ref = main + (0 if bias is None else bias.astype(np.float64))
    tol = (4 * np.abs(main) + np.abs(ref)) * 2.0 ** -24 + U[dtype] * np.abs(ref) * (1 + 2.0 ** -8)
    if dtype == "float16":
        tol = tol + 2.0 ** -25
    got = Y.double().cpu().numpy()
    assert got.shape == ref.shape
    worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)) if got.size else 0.0
    assert worst <= 1.0, worst


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("t,k", [(1, 1), (1, 4096), (3, 5), (7, 1000), (33, 1024), (2, 14336), (130, 333), (1, 100003)])
def test_codes_of_activations_are_equal_to_the_definition(bk, t, k, dtype):
    x = _values(np.random.default_rng(t * 1000 + k), t, k, dtype)
    c, s = bk.quantize_tokens(x)
    rc, rs = _reference_codes(x)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(c.cpu().numpy(), rc)


def test_codes_at_ties_zero_rows_and_tiny_rows(bk):
    import torch

    x = np.zeros((6, 256), dtype=np.float32)
    x[0, :255] = np.arange(255) - 127  # scale 1: codes are the values
    x[1, 0] = 127
    x[1, 1:129] = np.arange(128) - 63.5  # ties
    x[2] = 0
    x[3, :3] = [1e-45, -1e-45, 0]  # the scale underflows to 0
    x[4, :4] = [1e-40, -3e-41, 5e-42, 0]  # a subnormal scale
    x[5, :4] = [3e38, -1e38, 1e37, 1.0]
    x = torch.from_numpy(x).cuda()
    c, s = bk.quantize_tokens(x)
    rc, rs = _reference_codes(x)
    rc[rs == 0] = 0
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(c.cpu().numpy(), rc)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_is_not_finite_is_nan_and_leaves_the_others_alone(bk, bad):
    import torch

    rng = np.random.default_rng(5)
    for t in (1, 3, 40, 300):
        x, v = _values(rng, t, 200, "bfloat16"), _codes(rng, 70, 200)
        w = torch.rand(70, device="cuda")
        clean, _ = bk.int8_matmul(x, v, w)
        x[t // 2, 77] = bad
        c, s = bk.quantize_tokens(x)
        assert torch.isnan(s[t // 2]) and not c[t // 2].any() and int(torch.isnan(s).sum()) == 1
        y, st = bk.int8_matmul(x, v, w)
        assert int(st.item()) == 0
        assert torch.isnan(y[t // 2]).all()
        rest = torch.arange(t, device="cuda") != t // 2
        assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (1, 4096, 512), (2, 100, 37), (5, 3, 1000), (8, 4096, 130), (9, 4099, 65),
                                   (16, 64, 128), (17, 1040, 129), (33, 2064, 300), (64, 4096, 256), (65, 1000, 1999),
                                   (130, 272, 257), (200, 14336, 140), (257, 128, 64), (513, 1025, 200),
                                   (1100, 512, 384), (2049, 160, 1000)])
def test_product_of_values(bk, t, k, n, dtype):
    import torch

    rng = np.random.default_rng(t + k + n)
    x, v = _values(rng, t, k, dtype), _codes(rng, n, k)
    w = torch.from_numpy(rng.uniform(1e-4, 1e-3, n).astype(np.float32)).cuda()
    bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda() if n % 2 else None
    y, st = bk.int8_matmul(x, v, w, bias=bias)
    assert int(st.item()) == 0 and y.dtype == x.dtype
    rc, rs = _reference_codes(x)
    _check(y, rc, rs, v.cpu().numpy(), w.cpu().numpy(), None if bias is None else bias.cpu().numpy(), dtype)


@pytest.mark.parametrize("t", [1, 7, 8, 9, 31, 100, 300, 1500])
@pytest.mark.parametrize("k,n", [(4096, 256), (1041, 77)])
def test_product_of_given_codes_and_every_output_type(bk, t, k, n):
    import torch

    rng = np.random.default_rng(t * k)
    c, v = _codes(rng, t, k), _codes(rng, n, k)
    s = torch.from_numpy(rng.uniform(0.01, 0.1, t).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.uniform(1e-5, 1e-4, n).astype(np.float32)).cuda()
    for dtype in ("float32", "float16", "bfloat16"):
        y, st = bk.int8_matmul(c, v, w, x_scales=s, dtype=getattr(torch, dtype))
        assert int(st.item()) == 0
        _check(y, c.cpu().numpy(), s.cpu().numpy(), v.cpu().numpy(), w.cpu().numpy(), None, dtype)
    assert bk.int8_matmul(c, v, w, x_scales=s)[0].dtype == torch.float32


@pytest.mark.parametrize("t", [1, 8, 24, 140, 1100])
@pytest.mark.parametrize("k", [1024, 1025, 14336, 131056])
def test_sums_stay_exact_at_the_largest_codes(bk, t, k):
    """All codes -128, and a last column of ones: sums up to 2^31 - 2^18 whose lowest bits count."""
    import torch

    n = 136
    c = torch.full((t, k), -128, dtype=torch.int8, device="cuda")
    v = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    v[:, -1] = torch.arange(n, device="cuda").to(torch.int8) - 60
    ones_t, ones_n = torch.ones(t, device="cuda"), torch.ones(n, device="cuda")
    total = 16384 * (k - 1) - 128 * v[:, -1].double()
    y, st = bk.int8_matmul(c, v, ones_n, x_scales=ones_t)
    assert int(st.item()) == 0
    assert torch.equal(y, total.float().expand(t, n))


@pytest.mark.parametrize("t", [1, 12, 90, 1200])
def test_strided_and_unaligned_operands(bk, t):
    import torch

    rng = np.random.default_rng(t)
    k, n = 192, 96
    wide_x, wide_v = _values(rng, t, k + 37, "bfloat16"), _codes(rng, n, k + 21)
    w = torch.rand(n, device="cuda")
    for off in (0, 1, 8, 16):
        x, v = wide_x[:, off : off + k], wide_v[:, off : off + k]
        y, _ = bk.int8_matmul(x, v, w)
        assert torch.equal(y, bk.int8_matmul(x.contiguous(), v.contiguous(), w)[0])
        c, s = bk.quantize_tokens(x)
        c2, s2 = bk.quantize_tokens(x.contiguous())
        assert torch.equal(c, c2) and torch.equal(s, s2)
    c = _codes(rng, t, k + 9)[:, 3 : 3 + k]
    s = torch.rand(t, device="cuda")
    assert torch.equal(bk.int8_matmul(c, v, w, x_scales=s)[0],
                       bk.int8_matmul(c.contiguous(), v.contiguous(), w, x_scales=s)[0])


def test_packed_codes_of_a_quantized_layer(bk):
    """From the solve: codes of quantize_range, through pack_codes, into the product."""
    import torch

    rng = np.random.default_rng(11)
    m, n, t = 72, 96, 20
    W = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).cuda()
    A = torch.from_numpy(np.cov(rng.standard_normal((n, 4 * n))).astype(np.float32)).cuda()
    LA, LB, _ = bk.prepare(A, torch.eye(m, device="cuda"))
    scales = bk.row_scales(W, -127, 127)
    V, Wq, st = bk.quantize_range(W, LA, None, scales, -127, 127)
    x = _values(rng, t, n, "float32")
    y8, _ = bk.int8_matmul(x, V.to(torch.int8), scales)
    yp, _ = bk.int8_matmul(x, bk.pack_codes(V, 8), scales)
    assert int(st.item()) == 0 and torch.equal(y8, yp)
    exact = x.double() @ Wq.double().t()
    # what the activations' own codes may lose: half a step of each entry
    s = x.abs().amax(1).double() / 127
    assert bool(((y8.double() - exact).abs() <= 0.51 * s[:, None] * Wq.double().abs().sum(1)).all())


def test_no_tokens_and_another_stream(bk):
    import torch

    rng = np.random.default_rng(3)
    v, w = _codes(rng, 40, 64), torch.rand(40, device="cuda")
    y, st = bk.int8_matmul(torch.empty((0, 64), device="cuda"), v, w)
    assert y.shape == (0, 40) and int(st.item()) == 0
    c, s = bk.quantize_tokens(torch.empty((0, 64), device="cuda"))
    assert c.shape == (0, 64) and s.shape == (0,)
    side = torch.cuda.Stream()
    for t in (1, 50, 1300):
        x = _values(rng, t, 64, "float16")
        here, _ = bk.int8_matmul(x, v, w)
        side.wait_stream(torch.cuda.current_stream())
        there, _ = bk.int8_matmul(x, v, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(here, there)


def test_results_repeat(bk):
    import torch

    rng = np.random.default_rng(4)
    for t in (1, 40, 500):
        x, v, w = _values(rng, t, 5000, "bfloat16"), _codes(rng, 300, 5000), torch.rand(300, device="cuda")
        first = bk.int8_matmul(x, v, w)[0]
        for _ in range(5):
            assert torch.equal(first, bk.int8_matmul(x, v, w)[0])


def test_refusals(bk):
    import torch

    x, v, w = torch.ones((4, 64), device="cuda"), torch.ones((8, 64), dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    c, s = bk.quantize_tokens(x)
    for call in (lambda: bk.int8_matmul(x.cpu(), v, w), lambda: bk.int8_matmul(x, v.cpu(), w),
                 lambda: bk.int8_matmul(x, v[:, :32], w), lambda: bk.int8_matmul(x, v, w[:4]),
                 lambda: bk.int8_matmul(x, v, w.double()), lambda: bk.int8_matmul(x.double(), v, w),
                 lambda: bk.int8_matmul(c, v, w), lambda: bk.int8_matmul(x, v, w, x_scales=s),
                 lambda: bk.int8_matmul(c, v, w, x_scales=s[:2]), lambda: bk.int8_matmul(x, v.float(), w),
                 lambda: bk.int8_matmul(x, v, w, bias=w[:3]), lambda: bk.int8_matmul(x, v, w, dtype=torch.float64),
                 lambda: bk.int8_matmul(x[0], v, w), lambda: bk.int8_matmul(x.t()[:4], v[:, :4], w),
                 lambda: bk.int8_matmul(x[:1].expand(4, 64), v, w), lambda: bk.quantize_tokens(x.to(torch.int32)),
                 lambda: bk.quantize_tokens(x[:, :0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):  # 2^14 K would pass 2^31
        k = 1 << 17
        bk.int8_matmul(torch.zeros((1, k), device="cuda"), torch.zeros((1, k), dtype=torch.int8, device="cuda"), w[:1])
