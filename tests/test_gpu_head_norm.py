"""Norms of queries and keys for each head with the position rotation
(bakron_head_norm_rotary) and their gradients, against fp64.

In units of 2^-24.  A head's mean square is a sum of at most 37 roundings deep
(D / 32 values a lane, five exchanges, the mean, eps), so 1 / sqrt of it is off
by at most 19 + 1 of them, a normed value by 3 more.  An angle is off by less than 1 from its
rounding (at most an eighth of a turn, in fp32), its cosine and sine by 4 more
(two units in the last place); a turned value has one rounding more.  So
|error| <= 32 * 2^-24 (|n_a| + |n_b|), plus the output's own rounding u |y|.  Backward the two
sums, of squares and of g u, take part: 64 * 2^-24 of the sum of the terms' magnitudes.  Weight gradients are sums of
blocks' sums in a tree at most 128 deep for the sizes here.  Beyond |p f| = 2^28 the share of a turn, exact to
|p f| 2^-54 turns, adds 2 pi times that."""

import math

import numpy as np
import pytest

from test_gpu_int8_matmul import U, bk  # noqa: F401

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def _inputs(rng, t, hq, hk, d, dtype, extra=0, pad=0):
    """Queries and keys as views into one buffer of tokens, heads of d + pad values, `extra` heads behind."""
    import torch

    heads = hq + hk + extra
    x = rng.standard_normal((t, heads, d + pad)) * np.where(rng.random(heads * (d + pad)).reshape(1, heads, -1) < 0.05, 6.0, 1.0)
    x = torch.from_numpy(x.astype(np.float32)).cuda().to(getattr(torch, dtype))
    return x[:, :hq, :d], x[:, hq : hq + hk, :d]


def _args(rng, t, d, r, base=10000.0, start=0):
    import torch

    f = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / max(r, 1))
    p = torch.arange(t, device="cuda") + start
    w = [torch.from_numpy((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)).cuda() for _ in range(2)]
    return p, f, w


def _pairs(r, pairs):
    import torch

    i = torch.arange(r // 2, device="cuda")
    return (i, i + r // 2) if pairs == "halves" else (2 * i, 2 * i + 1)


def _turned(x, p, f, pairs, back=False):
    """Rotation in fp64 and the sums of magnitudes that make up each value."""
    a, b = _pairs(2 * len(f), pairs)
    angle = p.double()[:, None, None] * f
    c, s = angle.cos(), angle.sin() * (-1 if back else 1)
    y, size = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    both = x[..., a].abs() + x[..., b].abs()
    size[..., a], size[..., b] = both, both
    return y, size


def _normed(x, w, eps):
    x = x.double()
    if w is None:
        return x
    return x * torch_rsqrt(x, eps) * w.double()


def torch_rsqrt(x, eps):
    return (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()


def _own(dtype):
    return U[dtype] * (1 + 2.0 ** -8), 2.0 ** -25 if dtype == "float16" else 1e-40


def _close(y, ref, size, dtype):
    u, least = _own(dtype)
    assert y.shape == ref.shape and y.is_contiguous()
    if y.numel():
        worst = float(((y.double() - ref).abs() / (32 * E * size + u * ref.abs() + least)).max())
        assert worst <= 1.0, worst


def _check(bk, q, k, p, f, qw, kw, pairs, dtype, eps=1e-6):  # noqa: F811
    out = bk.head_norm_rotary(q, k, p, f, qw, kw, eps, pairs)
    for y, x, w in zip(out, (q, k), (qw, kw)):
        if x is None:
            assert y is None
            continue
        n = _normed(x, w, eps)
        _close(y, *(_turned(n, p, f, pairs) if f is not None else (n, n.abs())), dtype)
    return out


SHAPES = [(1, 1, 1, 2, 2), (1, 32, 8, 128, 128), (3, 4, 1, 64, 64), (17, 7, 3, 80, 20), (33, 5, 2, 96, 48), (9, 3, 1, 77, 76),
          (130, 2, 2, 256, 64), (1000, 8, 2, 128, 128), (41, 2, 1, 512, 512), (11, 2, 1, 1024, 1024), (5, 3, 2, 1, 0),
          (700, 12, 4, 48, 16), (2600, 6, 2, 64, 32), (64, 1, 1, 400, 100), (21, 9, 9, 16, 16), (8, 2, 1, 513, 512), (13, 4, 2, 80, 40), (9, 3, 1, 96, 72), (7, 2, 2, 24, 8),
          (130, 3, 1, 72, 64)]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("t,hq,hk,d,r", SHAPES)
def test_norm_and_rotation(bk, t, hq, hk, d, r, pairs, dtype):  # noqa: F811
    rng = np.random.default_rng(t + d)
    q, k = _inputs(rng, t, hq, hk, d, dtype, extra=hk)
    p, f, (qw, kw) = _args(rng, t, d, r, start=1000 * (t % 7))
    if r == 0:
        p = f = None
    out = _check(bk, q, k, p, f, qw, kw, pairs, dtype)
    # a side alone, and without its weight
    import torch

    assert torch.equal(bk.head_norm_rotary(k, None, p, f, kw, None, 1e-6, pairs)[0], out[1])
    _check(bk, q, k, p, f, None, kw, pairs, dtype)
    _check(bk, q, k, None, None, qw, None, pairs, dtype)


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_strides_orders_and_alignment(bk, pairs):  # noqa: F811
    """Heads before tokens, heads with a gap, tokens in reverse order, a lone token of any stride, values off 16 bytes."""
    import torch

    rng = np.random.default_rng(7)
    for t, hq, hk, d in ((40, 4, 2, 64), (1, 3, 1, 128), (6, 5, 5, 48)):
        p, f, (qw, kw) = _args(rng, t, d, d // 2 // 16 * 16 + 16)
        for dtype in ("float32", "bfloat16"):
            for pad in (0, 1, 8):
                q, k = _inputs(rng, t, hq, hk, d, dtype, pad=pad)
                want = bk.head_norm_rotary(q.contiguous(), k.contiguous(), p, f, qw, kw, 1e-6, pairs)
                for a, b in ((q, k), (q.transpose(0, 1).contiguous().transpose(0, 1), k),
                             (q, torch.empty((hk, t, d + 3), dtype=k.dtype, device="cuda")[..., 3:].copy_(k.transpose(0, 1)).transpose(0, 1))):
                    got = bk.head_norm_rotary(a, b, p, f, qw, kw, 1e-6, pairs)
                    for x, y in zip(got, want):
                        # other variants sum a head's squares in another order: twice the bound of one
                        u, least = _own(dtype)
                        size = _turned(_normed(a if x is got[0] else b, qw if x is got[0] else kw, 1e-6), p, f, pairs)[1]
                        assert bool(((x.double() - y.double()).abs() <= 64 * E * size + 2 * u * y.double().abs() + 2 * least).all())
                one = q[:1].expand(t, hq, d)  # a token for all, each at its own position
                got = bk.head_norm_rotary(one, None, p, f, qw, None, 1e-6, pairs)[0]
                assert torch.equal(got, bk.head_norm_rotary(one.contiguous(), None, p, f, qw, None, 1e-6, pairs)[0]) or pad


def test_positions_of_any_size(bk):  # noqa: F811
    """Far, negative and repeated positions, frequencies above a turn for each position: against the angle in 200 bits."""
    import torch

    mpmath = pytest.importorskip("mpmath")
    rng = np.random.default_rng(9)
    d = 16
    p = torch.tensor([0, 1, 7, -1, -12345, 131071, 1 << 20, (1 << 31) - 1, (1 << 33) + 5, -(1 << 40) - 3, 7], device="cuda")
    f = torch.tensor([1.0, 0.1, 1e-4, 3.7, 6.283185307179586, 100.25, 0.0, -0.5], dtype=torch.float64, device="cuda")
    t = len(p)
    x = torch.from_numpy(rng.standard_normal((t, 2, d)).astype(np.float32)).cuda()
    for pairs in ("halves", "neighbours"):
        y = bk.head_norm_rotary(x, None, p, f, pairs=pairs)[0].double().cpu()
        a, b = (i.cpu() for i in _pairs(d, pairs))
        xc = x.double().cpu()
        with mpmath.workprec(200):
            for i in range(t):
                for j in range(len(f)):
                    angle = mpmath.mpf(int(p[i])) * mpmath.mpf(float(f[j]))
                    c, s = float(mpmath.cos(angle)), float(mpmath.sin(angle))
                    tol = 32 * E + 2 * math.pi * (abs(int(p[i]) * float(f[j])) * 2.0 ** -54 + abs(int(p[i])) * 2.0 ** -64)
                    for h in range(2):
                        u, v = float(xc[i, h, a[j]]), float(xc[i, h, b[j]])
                        assert abs(float(y[i, h, a[j]]) - (u * c - v * s)) <= tol * (abs(u) + abs(v))
                        assert abs(float(y[i, h, b[j]]) - (v * c + u * s)) <= tol * (abs(u) + abs(v))


def test_frequencies_that_are_not_finite(bk):  # noqa: F811
    """NaN in the values of their pairs, numbers in the others, at position 0 too."""
    import torch

    for d in (16, 18):
        f = torch.ones(d // 2, dtype=torch.float64, device="cuda")
        f[1], f[3] = float("inf"), float("nan")
        y = bk.head_norm_rotary(torch.ones((3, 2, d), device="cuda"), None, torch.arange(3, device="cuda"), f)[0]
        bad = torch.zeros(d, dtype=torch.bool, device="cuda")
        for i in (1, 3):
            bad[i] = bad[i + d // 2] = True
        assert torch.equal(torch.isnan(y), bad.expand_as(y))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("d", [64, 77])
def test_heads_of_zeros_and_not_finite(bk, d, dtype):  # noqa: F811
    """A head of zeros is zeros (its gradient too, but for 1 / sqrt(eps)); a NaN or an infinity stays within its head."""
    import torch

    rng = np.random.default_rng(d)
    q, _ = _inputs(rng, 20, 4, 0, d, dtype)
    q = q.clone()
    p, f, (w, _) = _args(rng, 20, d, 32)
    clean = bk.head_norm_rotary(q, None, p, f, w)[0]
    q[3, 1], q[4, 2, 5], q[5, 0, 7] = 0, float("nan"), float("inf")
    y = bk.head_norm_rotary(q, None, p, f, w)[0]
    assert not y[3, 1].any() and torch.isnan(y[4, 2]).all()
    assert not torch.isfinite(y[5, 0, 7])
    same = torch.ones((20, 4), dtype=torch.bool, device="cuda")
    for i, h in ((3, 1), (4, 2), (5, 0)):
        same[i, h] = False
    assert torch.equal(y[same], clean[same])
    zero = torch.zeros_like(q)
    assert torch.isnan(bk.head_norm_rotary(zero, None, p, f, w, eps=0.0)[0]).all()  # 0 * inf, as the formula has it


def _gradients(x, dy, p, f, w, eps, pairs):
    """dx, dw from the formula in fp64, with the sums of their terms' magnitudes."""
    dy = dy.double()
    dn, size = (dy, dy.abs()) if f is None else _turned(dy, p, f, pairs, back=True)
    if w is None:
        return dn, size, None, None
    x, w = x.double(), w.double()
    r = torch_rsqrt(x, eps)
    u, g = x * r, dn * w
    dx = (g - u * (g * u).mean(-1, keepdim=True)) * r
    m = (size * w.abs() + u.abs() * (size * w.abs() * u.abs()).mean(-1, keepdim=True)) * r
    return dx, m, (dn * u).sum((0, 1)), (size * u.abs()).sum((0, 1))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("t,hq,hk,d,r", SHAPES)
def test_gradients(bk, t, hq, hk, d, r, pairs, dtype):  # noqa: F811
    import torch

    rng = np.random.default_rng(t + d)
    q, k = _inputs(rng, t, hq, hk, d, dtype, extra=hk)
    dq, dk = _inputs(rng, t, hq, hk, d, dtype)
    p, f, (qw, kw) = _args(rng, t, d, r, start=77)
    if r == 0:
        p = f = None
    u, least = _own(dtype)
    for a, b in ((qw, kw), (None, kw), (qw, None), (None, None)):
        g = bk.head_norm_rotary_backward(dq, dk, q, k, p, f, a, b, 1e-6, pairs)
        for name, x, dy, w in (("Q", q, dq, a), ("K", k, dk, b)):
            dx, m, dw, dm = _gradients(x, dy, p, f, w, 1e-6, pairs)
            assert g[name].shape == dx.shape and g[name].dtype == x.dtype
            assert bool(((g[name].double() - dx).abs() <= 64 * E * m + u * dx.abs() + least).all())
            got = g[name.lower() + "_weight"]
            assert (got is None) == (w is None)
            if w is not None:
                assert bool(((got.double() - dw).abs() <= 128 * E * dm + 1e-40).all())
    alone = bk.head_norm_rotary_backward(dq, None, q, None, p, f, qw, None, 1e-6, pairs)
    both = bk.head_norm_rotary_backward(dq, dk, q, k, p, f, qw, kw, 1e-6, pairs)
    assert alone["K"] is None and alone["k_weight"] is None and torch.equal(alone["Q"], both["Q"])


def test_gradients_against_differences(bk):  # noqa: F811
    """Central differences of <dY, y> in fp64: h^2 = 1e-10 of its third derivative, below a tenth of the bound."""
    import torch

    rng = np.random.default_rng(1)
    t, h, d, r, eps = 30, 3, 64, 32, 1e-5
    q, _ = _inputs(rng, t, h, 0, d, "float32")
    dq, _ = _inputs(rng, t, h, 0, d, "float32")
    p, f, (w, _) = _args(rng, t, d, r, start=5)
    for pairs in ("halves", "neighbours"):
        g = bk.head_norm_rotary_backward(dq, None, q, None, p, f, w, None, eps, pairs)
        _, m, _, dm = _gradients(q, dq, p, f, w, eps, pairs)

        def loss(x, w):
            return float((_turned(x * torch_rsqrt(x, eps) * w, p, f, pairs)[0] * dq.double()).sum())

        step = 1e-5
        x, v = q.double(), w.double()
        a = torch.randn(x.shape, dtype=torch.float64, device="cuda")
        b = torch.randn(d, dtype=torch.float64, device="cuda")
        slope = (loss(x + step * a, v) - loss(x - step * a, v)) / (2 * step)
        assert abs(slope - float((g["Q"].double() * a).sum())) <= 70 * E * float((m * a.abs()).sum())
        slope = (loss(x, v + step * b) - loss(x, v - step * b)) / (2 * step)
        assert abs(slope - float((g["q_weight"].double() * b).sum())) <= 128 * E * float((dm * b.abs()).sum())


def test_the_rotation_alone_is_undone_by_its_gradient(bk):  # noqa: F811
    import torch

    rng = np.random.default_rng(2)
    q, k = _inputs(rng, 50, 3, 1, 80, "float32")
    p, f, _ = _args(rng, 50, 80, 64)
    yq, yk = bk.head_norm_rotary(q, k, p, f)
    g = bk.head_norm_rotary_backward(yq, yk, q, k, p, f)
    for back, x in ((g["Q"], q), (g["K"], k)):
        size = _turned(x.double(), p, f, "halves")[1]
        assert bool(((back - x).abs().double() <= 2 * 64 * E * size).all())


def test_no_tokens_no_heads_and_another_stream(bk):  # noqa: F811
    import torch

    rng = np.random.default_rng(3)
    p, f, (qw, kw) = _args(rng, 0, 64, 64)
    q, k = _inputs(rng, 0, 4, 2, 64, "bfloat16")
    a, b = bk.head_norm_rotary(q, k, p, f, qw, kw)
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
    g = bk.head_norm_rotary_backward(a, b, q, k, p, f, qw, kw)
    assert g["Q"].shape == (0, 4, 64) and not g["q_weight"].any() and not g["k_weight"].any()
    p, f, _ = _args(rng, 9, 64, 64)
    q, k = _inputs(rng, 9, 4, 0, 64, "bfloat16")
    want = bk.head_norm_rotary(q, None, p, f, qw)[0]
    y, none = bk.head_norm_rotary(q, k, p, f, qw, kw)
    assert torch.equal(y, want) and none.shape == (9, 0, 64)
    g = bk.head_norm_rotary_backward(y, none, q, k, p, f, qw, kw)
    assert not g["k_weight"].any() and torch.equal(g["Q"], bk.head_norm_rotary_backward(y, None, q, None, p, f, qw)["Q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = bk.head_norm_rotary(q, None, p, f, qw, stream=side)[0]
    g2 = bk.head_norm_rotary_backward(there, None, q, None, p, f, qw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(there, want) and torch.equal(g2["Q"], g["Q"]) and torch.equal(g2["q_weight"], g["q_weight"])


def test_keys_without_queries(bk):  # noqa: F811
    import torch

    rng = np.random.default_rng(8)
    for d in (64, 50):
        q, k = _inputs(rng, 70, 0, 3, d, "bfloat16")
        p, f, (qw, kw) = _args(rng, 70, d, 32)
        want = bk.head_norm_rotary(k, None, p, f, kw)[0]
        none, y = bk.head_norm_rotary(q, k, p, f, qw, kw)
        assert none.shape == (70, 0, d) and torch.equal(y, want)
        g = bk.head_norm_rotary_backward(none, y, q, k, p, f, qw, kw)
        h = bk.head_norm_rotary_backward(y, None, k, None, p, f, kw)
        assert not g["q_weight"].any() and torch.equal(g["K"], h["Q"])
        # other blocks sum the weight's gradient: in another order
        size = _gradients(k, y, p, f, kw, 1e-6, "halves")[3]
        assert bool(((g["k_weight"] - h["q_weight"]).abs().double() <= 2 * 128 * E * size).all())


def test_offsets_beyond_32_bits(bk):  # noqa: F811
    """A token whose values lie more than 2^32 elements into the buffer."""
    import torch

    d, stride = 64, (1 << 31) + 64
    room = torch.empty(3 * stride, dtype=torch.bfloat16, device="cuda")
    q = room.as_strided((3, 2, d), (stride, d, 1))
    rng = np.random.default_rng(6)
    small, _ = _inputs(rng, 3, 2, 0, d, "bfloat16")
    q.copy_(small)
    p, f, (w, _) = _args(rng, 3, d, d)
    assert torch.equal(bk.head_norm_rotary(q, None, p, f, w)[0], bk.head_norm_rotary(small.contiguous(), None, p, f, w)[0])
    a = bk.head_norm_rotary_backward(q, None, q, None, p, f, w)
    b = bk.head_norm_rotary_backward(small.contiguous(), None, small.contiguous(), None, p, f, w)
    assert torch.equal(a["Q"], b["Q"]) and torch.equal(a["q_weight"], b["q_weight"])


def test_results_repeat(bk):  # noqa: F811
    import torch

    rng = np.random.default_rng(4)
    for t, d in ((3, 128), (5000, 64), (900, 77)):
        q, k = _inputs(rng, t, 6, 2, d, "bfloat16")
        p, f, (qw, kw) = _args(rng, t, d, d // 2 * 2)
        y = bk.head_norm_rotary(q, k, p, f, qw, kw)
        g = bk.head_norm_rotary_backward(*y, q, k, p, f, qw, kw)
        for _ in range(4):
            assert all(torch.equal(a, b) for a, b in zip(y, bk.head_norm_rotary(q, k, p, f, qw, kw)))
            again = bk.head_norm_rotary_backward(*y, q, k, p, f, qw, kw)
            assert all(torch.equal(g[i], again[i]) for i in g)


def test_refusals(bk):  # noqa: F811
    import torch

    q, k = torch.ones((4, 3, 16), device="cuda"), torch.ones((4, 1, 16), device="cuda")
    p, f, w = torch.arange(4, device="cuda"), torch.ones(8, dtype=torch.float64, device="cuda"), torch.ones(16, device="cuda")
    fwd, bwd = bk.head_norm_rotary, bk.head_norm_rotary_backward
    for call in (lambda: fwd(q.cpu(), k, p, f), lambda: fwd(q, k.cpu(), p, f), lambda: fwd(q[0], k, p, f),
                 lambda: fwd(q, k[:3], p, f), lambda: fwd(q, k[..., :8], p, f), lambda: fwd(q, k.half(), p, f),
                 lambda: fwd(q.double(), None, p, f), lambda: fwd(q, k, p[:3], f), lambda: fwd(q, k, p.int(), f),
                 lambda: fwd(q, k, p, f.float()), lambda: fwd(q, k, p, None), lambda: fwd(q, k, None, f),
                 lambda: fwd(q, k, p, torch.ones(9, dtype=torch.float64, device="cuda")), lambda: fwd(q, k, p, f, w[:8]),
                 lambda: fwd(q, k, p, f, w.half()), lambda: fwd(q, None, p, f, w, w), lambda: fwd(q, k, p, f, pairs="thirds"),
                 lambda: fwd(q.transpose(1, 2), None, p, f), lambda: fwd(torch.ones((4, 1, 1025), device="cuda"), None, None, None),
                 lambda: bwd(q, None, q, k, p, f), lambda: bwd(q, k, q, None, p, f), lambda: bwd(q[:, :2], k, q, k, p, f),
                 lambda: bwd(q, q, q, k, p, f), lambda: bwd(q, None, q, None, p, f, w, w)):
        with pytest.raises(ValueError):
            call()
    for eps in (-1.0, float("nan")):
        with pytest.raises(RuntimeError):
            fwd(q, k, p, f, w, eps=eps)
