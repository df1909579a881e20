"""e4m3 codes in blocks of 128 (bakron_quantize_blocks), the product of such
codes (bakron_fp8_matmul) and its gradients (bakron_fp8_matmul_backward).

Codes and scales are defined by single fp32 operations (a division, a
division, a product, a rounding), so they must be equal.

Products.  Products of two codes are exact in fp32.  The tensor cores add 32 of
them to a sum, four times for a block of 128; each of these additions may cut
what lies 2^-23 below the largest operand off each of its 33 terms, so a
block's sum is off by at most 4 * 33 * 2^-23 S, S the sum of the magnitudes of
its products.  Scaling takes at most three roundings of 2^-24 and each addition
of a block's sum one of 2^-24 of what has been summed, at most S scaled, in any
order: (blocks + 4) 2^-24 in all.  Then the bias (2^-24 of the result) and the
output type's own u (2^-24, 2^-11, 2^-8; fp16 adds half its smallest step,
2^-25)."""

import numpy as np
import pytest

from test_gpu_int8_matmul import U, _values, bk  # noqa: F401

pytestmark = pytest.mark.gpu


def _quantized(x, rows, cols):
    """The definition, in fp32 on the CPU: codes and scales."""
    import torch

    x = x.detach().float().cpu()
    t, k = x.shape
    r, c = -(-t // rows), -(-k // cols)
    full = torch.zeros((r * rows, c * cols))
    full[:t, :k] = x
    b = full.view(r, rows, c, cols)
    top = b.abs().amax((1, 3))
    scale = top / torch.tensor(448.0)
    live = (scale >= 2.0 ** -126) & torch.isfinite(top)
    inv = torch.where(live, 1 / scale, 0.0)
    q = torch.where(live[:, None, :, None], b * inv[:, None, :, None], 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    scale = torch.where(live, scale, torch.where(torch.isfinite(top), 0.0, float("nan")))
    return q.view(r * rows, c * cols)[:t, :k], scale


def _numbers(codes, scale, rows, cols):
    """What codes stand for, in fp64."""
    t, k = codes.shape
    return codes.double() * scale.double().repeat_interleave(rows, 0)[:t].repeat_interleave(cols, 1)[:, :k]


def _layer(bk, rng, n, k):  # noqa: F811
    import torch

    w = torch.from_numpy((rng.standard_normal((n, k)) * k ** -0.5 * rng.uniform(0.5, 2, (n, 1))).astype(np.float32)).cuda()
    return bk.quantize_blocks(w, (128, 128))


def _check(got, a, b, blocks, bias=None, dtype=None):
    """got against a b^T (+ bias), a and b the numbers of both operands' codes."""
    dtype = dtype or str(got.dtype).replace("torch.", "")
    ref, size = a @ b.t(), a.abs() @ b.abs().t()
    tol = size * (132 * 2.0 ** -23 + (blocks + 4) * 2.0 ** -24)
    if bias is not None:
        ref = ref + bias.double()
    tol = tol + ref.abs() * (2.0 ** -24 + U[dtype] * (1 + 2.0 ** -8)) + (2.0 ** -25 if dtype == "float16" else 0) + 1e-40
    assert got.shape == ref.shape
    worst = float(((got.double() - ref).abs() / tol).max()) if got.numel() else 0.0
    assert worst <= 1.0, worst


BLOCKS = [(1, 128), (128, 1), (128, 128)]


@pytest.mark.parametrize("block", BLOCKS)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("t,k", [(1, 1), (1, 4096), (3, 5), (127, 129), (128, 128), (129, 127), (300, 1000), (1, 100003),
                                 (1001, 7), (640, 272)])
def test_codes_are_equal_to_the_definition(bk, t, k, dtype, block):  # noqa: F811
    import torch

    x = _values(np.random.default_rng(t * 1000 + k), t, k, dtype)
    c, s = bk.quantize_blocks(x, block)
    rc, rs = _quantized(x, *block)
    assert c.dtype == torch.float8_e4m3fn and c.data_ptr() % 16 == 0 and (t == 1 or c.stride(0) % 16 == 0)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(c.cpu().view(torch.uint8), rc.contiguous().view(torch.uint8))


@pytest.mark.parametrize("block", BLOCKS)
def test_codes_of_ties_zeros_and_the_smallest_values(bk, block):  # noqa: F811
    """Every code comes back as itself, midpoints go to even codes, and blocks of zeros or of values so small that
    their reciprocal overflows are zeros with scale 0."""
    import torch

    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = codes[torch.isfinite(codes)]
    up = codes[(codes >= 0)].sort().values
    mid = (up[1:] + up[:-1]) / 2
    x = torch.zeros((6 * 128, 6 * 128))
    rows = [codes, mid, -mid, 1e-45 * codes.sign(), 3e35 * codes, 1e-35 * codes, 2.0 ** -126 * up]
    for i, r in enumerate(rows):
        for j in range(0, len(r), 127):  # a block's largest value sets its scale
            part = r[j : j + 127]
            at = 128 * (j // 127)
            x[i, at] = 448 if i < 3 else r.abs().max()
            x[i, at + 1 : at + 1 + len(part)] = part
    x[256:512, :128] = torch.randn((256, 128), generator=torch.Generator().manual_seed(1)) * 1e-40
    x[640:768, 128:] = x[:128, :640]
    for v in (x, x.t().contiguous()):
        c, s = bk.quantize_blocks(v.cuda(), block)
        rc, rs = _quantized(v, *block)
        assert torch.equal(s.cpu(), rs) and torch.equal(c.cpu().view(torch.uint8), rc.contiguous().view(torch.uint8))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("t", [1, 3, 100, 300])
def test_a_token_that_is_not_finite_is_nan_and_leaves_the_others_alone(bk, bad, t):  # noqa: F811
    import torch

    rng = np.random.default_rng(5)
    x, (v, w) = _values(rng, t, 200, "bfloat16"), _layer(bk, rng, 70, 200)
    clean, _ = bk.fp8_matmul(x, v, w)
    x[t // 2, 177] = bad
    for block in BLOCKS:
        c, s = bk.quantize_blocks(x, block)
        rc, rs = _quantized(x, *block)
        assert torch.equal(s.cpu().nan_to_num(nan=-1.0), rs.nan_to_num(nan=-1.0)) and int(torch.isnan(s).sum()) == 1
        assert torch.equal(c.cpu().view(torch.uint8), rc.contiguous().view(torch.uint8))
    y, st = bk.fp8_matmul(x, v, w)
    assert int(st.item()) == 0
    assert torch.isnan(y[t // 2]).all()
    rest = torch.arange(t, device="cuda") != t // 2
    assert torch.equal(y[rest], clean[rest])


# Few tokens of small and of large layers go different ways, and so do few and many outputs.
SHAPES = [(1, 200, 5000), (2, 6000, 24), (3, 520, 3001), (4, 3000, 513), (4, 4096, 4096), (2, 513, 31000), (1, 1, 1), (1, 4096, 512), (2, 100, 37), (5, 3, 1000), (8, 4096, 130), (9, 4099, 65), (16, 64, 128),
          (33, 2064, 300), (64, 4096, 256), (65, 1000, 1999), (128, 640, 264), (129, 640, 264), (200, 14336, 140),
          (257, 128, 64), (513, 1025, 200), (1100, 512, 384), (2049, 160, 1000), (2100, 200, 2601)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("t,k,n", SHAPES)
def test_product_of_values(bk, t, k, n, dtype):  # noqa: F811
    import torch

    rng = np.random.default_rng(t + k + n)
    x, (v, w) = _values(rng, t, k, dtype), _layer(bk, rng, n, k)
    bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda() if (n + t) % 2 else None
    y, st = bk.fp8_matmul(x, v, w, bias=bias)
    assert int(st.item()) == 0 and y.dtype == x.dtype
    c, s = _quantized(x, 1, 128)
    _check(y, _numbers(c.cuda(), s.cuda(), 1, 128), _numbers(v, w, 128, 128), -(-k // 128), bias)


@pytest.mark.parametrize("t", [1, 2, 3, 4, 7, 64, 65, 100, 300, 1500])
@pytest.mark.parametrize("k,n", [(4096, 256), (1041, 77), (640, 6000)])
def test_product_of_given_codes_and_every_output_type(bk, t, k, n):  # noqa: F811
    import torch

    rng = np.random.default_rng(t * k)
    x, (v, w) = _values(rng, t, k, "float32"), _layer(bk, rng, n, k)
    c, s = bk.quantize_blocks(x)
    a, b = _numbers(c, s, 1, 128), _numbers(v, w, 128, 128)
    for dtype in ("float32", "float16", "bfloat16"):
        y, st = bk.fp8_matmul(c, v, w, x_scales=s, dtype=getattr(torch, dtype))
        assert int(st.item()) == 0 and y.dtype == getattr(torch, dtype)
        _check(y, a, b, -(-k // 128))
    y = bk.fp8_matmul(c, v, w, x_scales=s)[0]
    assert y.dtype == torch.float32 and torch.equal(y, bk.fp8_matmul(x, v, w)[0])
    assert torch.equal(y, bk.fp8_matmul(c, v.view(torch.uint8), w, x_scales=s)[0])


@pytest.mark.parametrize("t", [1, 60, 128, 400])
@pytest.mark.parametrize("k", [128, 1024, 16384])
def test_large_codes_of_one_sign(bk, t, k):  # noqa: F811
    """All codes 448, scales of powers of two: every sum is a multiple of 448^2 below 2^24 of them, exact in fp32."""
    import torch

    n = 300
    c = torch.full((t, k), 448.0, device="cuda").to(torch.float8_e4m3fn)
    v = torch.full((n, k), -448.0, device="cuda").to(torch.float8_e4m3fn)
    blocks = k // 128
    s = (2.0 ** (torch.arange(t * blocks, device="cuda") % 3).float()).view(t, blocks)
    w = (2.0 ** (torch.arange(3 * blocks, device="cuda") % 2).float()).view(3, blocks)
    y, st = bk.fp8_matmul(c, v, w, x_scales=s)
    ref = -(448.0 ** 2) * 128 * (s.double() @ w.double().t())
    assert int(st.item()) == 0
    assert torch.equal(y.double(), ref.repeat_interleave(128, 1)[:, :n])


@pytest.mark.parametrize("t", [1, 3, 40, 90, 700])
def test_strided_and_unaligned_operands(bk, t):  # noqa: F811
    import torch

    rng = np.random.default_rng(t)
    k, n = 200, 96
    wide_x, wide_dy = _values(rng, t, k + 37, "bfloat16"), _values(rng, t, n + 19, "bfloat16")
    codes, w = _layer(bk, rng, n, k)
    c, s = bk.quantize_blocks(wide_x[:, :k].contiguous())

    def moved(a, off, pad):  # the same codes in other rows
        room = torch.zeros((a.shape[0], a.shape[1] + pad + off), dtype=torch.uint8, device="cuda")
        room[:, off : off + a.shape[1]] = a.view(torch.uint8) if a.is_contiguous() else a.contiguous().view(torch.uint8)
        return room.view(torch.float8_e4m3fn)[:, off : off + a.shape[1]]

    want = bk.fp8_matmul(wide_x[:, :k].contiguous(), codes, w)[0]
    want_c = bk.fp8_matmul(c, codes, w, x_scales=s)[0]
    for off, pad in ((0, 3), (1, 2), (3, 13), (16, 8), (8, 0)):
        v = moved(codes, off, pad)
        assert torch.equal(bk.fp8_matmul(wide_x[:, :k].contiguous(), v, w)[0], want)
        assert torch.equal(bk.fp8_matmul(moved(c, off, pad), v, w, x_scales=s)[0], want_c)
        x, dy = wide_x[:, off : off + k], wide_dy[:, off : off + n]
        for block in BLOCKS:
            a, b = bk.quantize_blocks(x, block), bk.quantize_blocks(x.contiguous(), block)
            assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
        g = bk.fp8_matmul_backward(dy, x, v, w, bias=True)[0]
        h = bk.fp8_matmul_backward(dy.contiguous(), x.contiguous(), codes, w, bias=True)[0]
        assert all(torch.equal(g[i], h[i]) for i in g)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (1, 300, 200), (7, 33, 65), (128, 128, 128), (130, 1000, 77), (513, 264, 1025),
                                   (777, 1000, 2055), (1030, 2600, 2100), (3000, 72, 40), (4500, 136, 260)])
def test_gradients(bk, t, k, n, dtype):  # noqa: F811
    import torch

    rng = np.random.default_rng(t + k + n)
    x, (v, w) = _values(rng, t, k, dtype), _layer(bk, rng, n, k)
    dy = (_values(rng, t, n, "float32") * torch.from_numpy(np.exp(rng.standard_normal((t, 1))).astype(np.float32)).cuda()).to(x.dtype)
    g, st = bk.fp8_matmul_backward(dy, x, v, w, bias=True)
    assert int(st.item()) == 0 and g["X"].dtype == g["W"].dtype == x.dtype and g["bias"].dtype == torch.float32

    def of(m, rows, cols):
        c, s = _quantized(m, rows, cols)
        return _numbers(c.cuda(), s.cuda(), rows, cols)

    _check(g["X"], of(dy, 1, 128), _numbers(v, w, 128, 128).t(), -(-n // 128))
    # A block of tokens has a scale for each row and each column: one rounding more, of 2^-24, in `blocks + 4`.
    _check(g["W"], of(dy, 128, 1).t(), of(x, 128, 1).t(), -(-t // 128) + 1)
    # 128 values in a tile (8, an exchange, 8 warps), then the tiles in their order
    tol = (18 + -(-t // 128)) * 2.0 ** -24 * dy.double().abs().sum(0) + 1e-40
    assert bool(((g["bias"].double() - dy.double().sum(0)).abs() <= tol).all())
    only, _ = bk.fp8_matmul_backward(dy, None, v, w)
    assert only["W"] is None and only["bias"] is None and torch.equal(only["X"], g["X"])


def test_gradients_against_differences(bk):  # noqa: F811
    """L = <dY, X V^T> is linear in X and in V: central differences in fp64 give its slope along a direction up to
    rounding, and the codes of dY and X are off by at most half a step (2^-4 of a value, or 2^-10 of its scale)."""
    import torch

    rng = np.random.default_rng(8)
    t, k, n = 300, 260, 200
    x, dy, (v, w) = _values(rng, t, k, "float32"), _values(rng, t, n, "float32"), _layer(bk, rng, n, k)
    g, _ = bk.fp8_matmul_backward(dy, x, v, w)
    V = _numbers(v, w, 128, 128)

    def loss(x, V):
        return float((dy.double() * (x @ V.t())).sum())

    def off(m, rows, cols):
        _, s = _quantized(m, rows, cols)
        return 2.0 ** -4 * m.double().abs() + 2.0 ** -10 * _numbers(torch.ones_like(m), s.cuda(), rows, cols)

    h = 1e-3
    for seed in range(3):
        d = torch.randn((t, k), dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        slope = (loss(x.double() + h * d, V) - loss(x.double() - h * d, V)) / (2 * h)
        tol = float((off(dy, 1, 128) @ V.abs() * d.abs()).sum()) * 1.01
        assert abs(slope - float((g["X"].double() * d).sum())) <= tol
        # and far inside of it: half steps of either sign do not add up
        assert abs(slope - float((g["X"].double() * d).sum())) <= 0.1 * tol
        e = torch.randn((n, k), dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(seed + 9))
        slope = (loss(x.double(), V + h * e) - loss(x.double(), V - h * e)) / (2 * h)
        a, b = off(dy, 128, 1), off(x, 128, 1)
        tol = float(((a.t() @ (x.double().abs() + b) + dy.double().abs().t() @ b) * e.abs()).sum()) * 1.01
        assert abs(slope - float((g["W"].double() * e).sum())) <= 0.1 * tol


@pytest.mark.parametrize("t", [100, 900])
def test_a_column_that_is_not_finite(bk, t):  # noqa: F811
    """An infinity in dY: its token's dX, its output's dW, and nothing else."""
    import torch

    rng = np.random.default_rng(t)
    k, n = 264, 150
    x, dy, (v, w) = _values(rng, t, k, "bfloat16"), _values(rng, t, n, "bfloat16"), _layer(bk, rng, n, k)
    clean, _ = bk.fp8_matmul_backward(dy, x, v, w)
    dy[t // 3, 55] = float("inf")
    g, st = bk.fp8_matmul_backward(dy, x, v, w)
    assert int(st.item()) == 0
    for name, row in (("X", t // 3), ("W", 55)):
        assert torch.isnan(g[name][row]).all()
        rest = torch.arange(g[name].shape[0], device="cuda") != row
        assert torch.equal(g[name][rest], clean[name][rest])


def test_no_tokens_and_another_stream(bk):  # noqa: F811
    import torch

    rng = np.random.default_rng(3)
    v, w = _layer(bk, rng, 40, 64)
    none = torch.empty((0, 64), device="cuda")
    y, st = bk.fp8_matmul(none, v, w)
    assert y.shape == (0, 40) and int(st.item()) == 0
    c, s = bk.quantize_blocks(none)
    assert c.shape == (0, 64) and s.shape == (0, 1)
    assert bk.fp8_matmul(c, v, w, x_scales=s)[0].shape == (0, 40)
    g, st = bk.fp8_matmul_backward(y, none, v, w, bias=True)
    assert g["X"].shape == (0, 64) and int(st.item()) == 0 and not g["W"].any() and not g["bias"].any()
    side = torch.cuda.Stream()
    for t in (1, 100, 1300):
        x = _values(rng, t, 64, "float16")
        here, _ = bk.fp8_matmul(x, v, w)
        grads, _ = bk.fp8_matmul_backward(here, x, v, w, bias=True)
        side.wait_stream(torch.cuda.current_stream())
        there, _ = bk.fp8_matmul(x, v, w, stream=side)
        grads2, _ = bk.fp8_matmul_backward(there, x, v, w, bias=True, stream=side)
        codes = bk.quantize_blocks(x, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(here, there) and all(torch.equal(grads[i], grads2[i]) for i in grads)
        assert torch.equal(codes[1], bk.quantize_blocks(x)[1])


def test_results_repeat(bk):  # noqa: F811
    import torch

    rng = np.random.default_rng(4)
    for t in (1, 70, 128, 500, 5000):
        x, (v, w) = _values(rng, t, 1000, "bfloat16"), _layer(bk, rng, 300, 1000)
        y = bk.fp8_matmul(x, v, w)[0]
        g = bk.fp8_matmul_backward(y, x, v, w, bias=True)[0]
        for _ in range(5):
            assert torch.equal(y, bk.fp8_matmul(x, v, w)[0])
            again = bk.fp8_matmul_backward(y, x, v, w, bias=True)[0]
            assert all(torch.equal(g[i], again[i]) for i in g)


def test_refusals(bk):  # noqa: F811
    import torch

    x, dy = torch.ones((4, 64), device="cuda"), torch.ones((4, 8), device="cuda")
    v, w = bk.quantize_blocks(torch.ones((8, 64), device="cuda"), (128, 128))
    c, s = bk.quantize_blocks(x)
    for call in (lambda: bk.fp8_matmul(x.cpu(), v, w), lambda: bk.fp8_matmul(x, v.cpu(), w), lambda: bk.fp8_matmul(x, v, w.cpu()),
                 lambda: bk.fp8_matmul(x, v[:, :32], w), lambda: bk.fp8_matmul(x, v, w[:0]), lambda: bk.fp8_matmul(x, v, w.double()),
                 lambda: bk.fp8_matmul(x.double(), v, w), lambda: bk.fp8_matmul(c, v, w), lambda: bk.fp8_matmul(x, v, w, x_scales=s),
                 lambda: bk.fp8_matmul(c, v, w, x_scales=s[:2]), lambda: bk.fp8_matmul(x, v.float(), w),
                 lambda: bk.fp8_matmul(x, v.to(torch.float8_e5m2), w), lambda: bk.fp8_matmul(x, v, w, bias=s[:3, 0]),
                 lambda: bk.fp8_matmul(x, v, w, dtype=torch.float64), lambda: bk.fp8_matmul(x[0], v, w),
                 lambda: bk.fp8_matmul(x.t()[:4], v[:, :4], w), lambda: bk.fp8_matmul(x[:1].expand(4, 64), v, w),
                 lambda: bk.fp8_matmul(x, v[:0], w), lambda: bk.quantize_blocks(x.to(torch.int32)),
                 lambda: bk.quantize_blocks(x[:, :0]), lambda: bk.quantize_blocks(x, (1, 64)), lambda: bk.quantize_blocks(x, (2, 128)),
                 lambda: bk.fp8_matmul_backward(dy, x[:3], v, w), lambda: bk.fp8_matmul_backward(dy[:, :7], x, v, w),
                 lambda: bk.fp8_matmul_backward(dy.half(), x, v, w), lambda: bk.fp8_matmul_backward(dy, x, v, w[0]),
                 lambda: bk.fp8_matmul_backward(dy, x, v[0], w), lambda: bk.fp8_matmul_backward(dy.cpu(), x, v, w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):  # K beyond 2^20
        k = (1 << 20) + 128
        bk.fp8_matmul(torch.zeros((1, k), device="cuda"), torch.zeros((1, k), dtype=torch.uint8, device="cuda"),
                      torch.zeros((1, k // 128), device="cuda"))
