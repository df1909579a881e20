"""Cross entropy over a vocabulary and its gradients
(bakron_linear_cross_entropy, bakron_linear_cross_entropy_grad), against fp64.

Tolerances.  A logit is a sum of D exact products in fp32: within
e = (2 D + 16) 2^-24 sum_d |h_d w_d| of its value (the sequential bound,
doubled for the order inside a tensor-core instruction).  lse moves by at most
the largest e of its row, plus the sum's own roundings: at most 1024 additions
along any path and an exponential good to 2^-21, 2^-13 in all, and 2^-22 of
lse and of the logits themselves.  An entry of G is within a relative
2 e + 2^-13 of p before it is rounded to 16 bits; on its way it may be held as
a 16-bit logarithm (step 2^-11, 2^-12 of p at most) that ends 2^-31 below its
row's largest, and is then rounded to the inputs' type, u = 2^-11 (fp16) or
2^-8 (bf16).  The gradients' sums (over V or T terms) add (2 n + 16) 2^-24 of
their magnitudes and the output's own u (fp16: and 2^-24, its smallest step).
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


@pytest.fixture(scope="module")
def bk():
    import torch

    import kronecker_hessian_gptq_gb300 as bk
    from kronecker_hessian_gptq_gb300 import build as b

    b.build()
    bk.load_library()
    torch.cuda.init()
    return bk


def _make(t, d, v, dtype, seed=0, spread=1.0):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed + t + 7 * d + 13 * v)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    w = (rand(v, d) * d ** -0.5).to(getattr(torch, dtype))
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    h = (spread * (rand(t, d) + 3 * torch.rand((t, 1), generator=gen, device="cuda") * w[y].float())).to(w.dtype)
    if t > 2:
        y[torch.rand(t, generator=gen, device="cuda") < 0.2] = -100
    return h, w, y


def _reference(h, w, y, coef=None):
    """fp64 loss, lse, gradients and the magnitudes their errors are measured by."""
    import torch

    h, w = h.double(), w.double()
    t, (v, d) = len(h), w.shape
    x = h @ w.t()
    e = (2 * d + 16) * 2.0 ** -24 * (h.abs() @ w.abs().t())
    lse = torch.logsumexp(x, 1)
    has = (y >= 0) & (y < v)
    at = y.clamp(0, v - 1)[:, None]
    right = x.gather(1, at)[:, 0]
    loss = torch.where(has, lse - right, 0.0)
    etol = e.amax(1) + 2.0 ** -13 + 2.0 ** -22 * (lse.abs() + x.abs().amax(1))
    ltol = torch.where(has, etol + e.gather(1, at)[:, 0], 0.0)
    if coef is None:
        coef = has.double() / has.sum().clamp(min=1)
    coef = torch.where(has, coef.double(), 0.0)[:, None]
    p = torch.exp(x - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, at, has.double()[:, None])
    g = coef * (p - hot)
    return {"loss": (loss, ltol), "lse": (lse, etol), "g": g, "coef": coef,
            "gerr": coef.abs() * (p * (2 * e.amax(1, keepdim=True) + 2.0 ** -13 + 2.0 ** -12) + 2.0 ** -31)}


def _close(got, ref, tol):
    worst = float(((got.double() - ref).abs() / (tol + 1e-300)).max()) if got.numel() else 0.0
    assert worst <= 1.0, worst


def _check_gradients(dh, dw, r, h, w, dtype):
    h, w, g = h.double(), w.double(), r["g"]
    err = r["gerr"] + U[dtype] * (g.abs() + r["gerr"])
    small = 2.0 ** -24 if dtype == "float16" else 1e-38
    for got, a, b, e in ((dh, g, w, err), (dw, g.t(), h, err.t())):
        ref = a @ b
        n = a.shape[1]
        tol = e @ b.abs() + (2 * n + 16) * 2.0 ** -24 * ((a.abs() + e) @ b.abs())
        _close(got, ref, tol + U[dtype] * (ref.abs() + tol) + small)


SHAPES = [(1, 8, 2), (1, 64, 1000), (2, 4096, 300), (3, 5, 7), (7, 100, 1), (17, 72, 513), (64, 128, 4096), (129, 256, 1999),
          (300, 64, 260), (513, 40, 777), (33, 1000, 5003), (257, 520, 12345), (16, 264, 128), (1030, 16, 300)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("t,d,v", SHAPES)
def test_loss_and_gradients(bk, t, d, v, dtype):
    h, w, y = _make(t, d, v, dtype)
    r = _reference(h, w, y)
    loss, lse, st = bk.linear_cross_entropy(h, w, y)
    assert int(st.item()) == 0
    _close(loss, *r["loss"])
    _close(lse, *r["lse"])
    loss2, lse2, dh, dw, st = bk.linear_cross_entropy_grad(h, w, y)
    assert int(st.item()) == 0 and dh.dtype == dw.dtype == h.dtype
    _close(loss2, *r["loss"])
    _close(lse2, *r["lse"])
    _check_gradients(dh, dw, r, h, w, dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_more_tokens_than_one_piece_holds(bk, dtype):
    """A vocabulary so large that the tokens are taken in several pieces."""
    h, w, y = _make(2600, 16, 200003, dtype)
    part = slice(1000, 1100)
    loss, lse, dh, dw, st = bk.linear_cross_entropy_grad(h, w, y)
    assert int(st.item()) == 0
    import torch

    has = y >= 0
    coef = has.double() / has.sum()
    dwr = torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    dwe = torch.zeros_like(dwr)
    for lo in range(0, 2600, 200):
        q = slice(lo, min(lo + 200, 2600))
        r = _reference(h[q], w, y[q], coef[q])
        _close(loss[q], *r["loss"])
        _close(lse[q], *r["lse"])
        e = r["gerr"] + U[dtype] * (r["g"].abs() + r["gerr"])
        hd = h[q].double()
        ref = r["g"] @ w.double()
        tol = e @ w.double().abs() + (2 * w.shape[0] + 16) * 2.0 ** -24 * ((r["g"].abs() + e) @ w.double().abs())
        _close(dh[q], ref, tol + U[dtype] * (ref.abs() + tol) + 2.0 ** -24)
        dwr += r["g"].t() @ hd
        dwe += e.t() @ hd.abs() + (2 * 2600 + 16) * 2.0 ** -24 * (r["g"].abs().t() @ hd.abs())
    _close(dw, dwr, dwe + U[dtype] * (dwr.abs() + dwe) + 2.0 ** -24)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("t,d,v", [(5, 48, 300), (140, 64, 1000)])
def test_given_coefficients(bk, t, d, v, dtype):
    """Coefficients of both signs, some of them zero (small ones in fp16 fall under its smallest step and are excused)."""
    import torch

    h, w, y = _make(t, d, v, dtype)
    coef = torch.randn(t, device="cuda")
    coef[::4] = 0
    r = _reference(h, w, y, coef)
    _, _, dh, dw, st = bk.linear_cross_entropy_grad(h, w, y, coef=coef)
    assert int(st.item()) == 0
    _check_gradients(dh, dw, r, h, w, dtype)
    assert not dh[::4].any()
    zero = bk.linear_cross_entropy_grad(h, w, y, coef=torch.zeros(t, device="cuda"))
    assert not zero[2].any() and not zero[3].any()


@pytest.mark.parametrize("spread", [0.0, 30.0, 200.0])
def test_flat_and_peaked_logits(bk, spread):
    h, w, y = _make(70, 128, 900, "bfloat16", spread=spread)
    r = _reference(h, w, y)
    loss, lse, dh, dw, st = bk.linear_cross_entropy_grad(h, w, y)
    assert int(st.item()) == 0
    _close(loss, *r["loss"])
    _close(lse, *r["lse"])
    _check_gradients(dh, dw, r, h, w, "bfloat16")


@pytest.mark.parametrize("t", [1, 3, 150])
def test_no_target_anywhere(bk, t):
    import torch

    h, w, _ = _make(t, 64, 400, "bfloat16")
    y = torch.full((t,), -1, device="cuda")
    loss, lse, dh, dw, st = bk.linear_cross_entropy_grad(h, w, y)
    assert int(st.item()) == 0 and not loss.any() and not dh.any() and not dw.any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("t", [1, 140])
def test_a_target_beyond_the_vocabulary_is_reported_and_left_out(bk, t):
    import torch

    h, w, y = _make(t, 64, 400, "float16")
    y[t // 2] = 400
    left = y.clone()
    left[t // 2] = -1
    got, ref = bk.linear_cross_entropy_grad(h, w, y), bk.linear_cross_entropy_grad(h, w, left)
    assert int(got[4].item()) == 8 and int(ref[4].item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(got[:4], ref[:4]))
    assert int(bk.linear_cross_entropy(h, w, y)[2].item()) == 8


@pytest.mark.parametrize("t", [2, 140])
def test_a_token_that_is_not_finite_keeps_to_its_row(bk, t):
    import torch

    h, w, y = _make(t, 64, 400, "bfloat16")
    y[0], y[1] = 3, 5
    clean = bk.linear_cross_entropy(h, w, y)
    h[1, 2] = float("nan")
    loss, lse, dh, dw, _ = bk.linear_cross_entropy_grad(h, w, y)
    rest = torch.arange(t, device="cuda") != 1
    assert torch.isnan(loss[1]) and torch.isnan(lse[1]) and torch.isnan(dh[1]).all() and torch.isnan(dw).any()
    assert torch.equal(loss[rest], clean[0][rest]) and torch.isfinite(dh[rest]).all()


def test_gradients_against_differences(bk):
    """Central differences of the fp64 mean loss along random directions."""
    import torch

    h, w, y = _make(40, 96, 500, "float16")
    r = _reference(h, w, y)
    has = y >= 0
    _, _, dh, dw, _ = bk.linear_cross_entropy_grad(h, w, y)

    def mean(h, w):
        x = h @ w.t()
        return float((torch.logsumexp(x, 1) - x.gather(1, y.clamp(min=0)[:, None])[:, 0])[has].mean())

    gen = torch.Generator(device="cuda").manual_seed(1)
    err = r["gerr"] + U["float16"] * (r["g"].abs() + r["gerr"])
    for got, at, e in ((dh, h, err @ w.double().abs()), (dw, w, err.t() @ h.double().abs())):
        step = torch.randn(at.shape, generator=gen, device="cuda", dtype=torch.float64)
        up, down = at.double() + 1e-5 * step, at.double() - 1e-5 * step
        slope = (mean(up, w.double()) - mean(down, w.double())) / 2e-5 if at is h else (mean(h.double(), up) - mean(h.double(), down)) / 2e-5
        tol = float((step.abs() * (1.1 * e + U["float16"] * got.double().abs() + 2.0 ** -24)).sum())
        assert abs(float((got.double() * step).sum()) - slope) <= tol + 1e-7


def test_strides_and_alignment(bk):
    import torch

    for t in (2, 140):
        h, w, y = _make(t, 300, 600, "bfloat16")
        for off, d in ((0, 256), (8, 256), (1, 256), (3, 250)):
            hs, ws = h[:, off : off + d], w[:, off : off + d]
            got, ref = bk.linear_cross_entropy_grad(hs, ws, y), bk.linear_cross_entropy_grad(hs.contiguous(), ws.contiguous(), y)
            assert all(torch.equal(a, b) for a, b in zip(got[:4], ref[:4]))
            assert torch.equal(bk.linear_cross_entropy(hs, ws, y)[0], bk.linear_cross_entropy(hs.contiguous(), ws.contiguous(), y)[0])


def test_no_tokens_another_stream_and_repeats(bk):
    import torch

    h, w, y = _make(0, 64, 100, "bfloat16")
    loss, lse, dh, dw, st = bk.linear_cross_entropy_grad(h, w, y)
    assert loss.shape == lse.shape == (0,) and dh.shape == (0, 64) and not dw.any() and int(st.item()) == 0
    h, w, y = _make(600, 200, 3001, "bfloat16")
    first = bk.linear_cross_entropy_grad(h, w, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = bk.linear_cross_entropy_grad(h, w, y, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, there))


def test_refusals(bk):
    import torch

    h, w, y = _make(6, 64, 100, "bfloat16")
    for call in (lambda: bk.linear_cross_entropy(h.float(), w.float(), y), lambda: bk.linear_cross_entropy(h, w.half(), y),
                 lambda: bk.linear_cross_entropy(h, w[:, :32], y), lambda: bk.linear_cross_entropy(h, w, y[:3]),
                 lambda: bk.linear_cross_entropy(h, w, y.int()), lambda: bk.linear_cross_entropy(h.cpu(), w, y),
                 lambda: bk.linear_cross_entropy(h, w[:0], y), lambda: bk.linear_cross_entropy(h.t(), w, y),
                 lambda: bk.linear_cross_entropy_grad(h, w, y, coef=torch.ones(6)),
                 lambda: bk.linear_cross_entropy_grad(h, w, y, coef=torch.ones(5, device="cuda"))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("t,d,v", [(20, 4096, 1000), (5, 4096, 8192), (130, 3000, 777)])
def test_log_sums_of_few_large_logits(bk, t, d, v, dtype):
    """Targets far above the rest, in a small vocabulary: lse is little else
    than the target's logit, so an error of its sum does not average out.  Sums
    that round towards zero every 16 terms lose half a unit (2^-24) of the sum
    so far each time, which is on average half of what it ends as: 2^-26 of
    the logit for every 16 terms.  Restarted every 512 terms that is 4.8e-7;
    over 4096 it would be 3.8e-6.  Twice the former, with 2^-22 for the
    exponentials' sum and the logarithm, is allowed over all tokens."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(t + d + v)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    w = (rand(v, d) * d ** -0.5).to(getattr(torch, dtype))
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    h = (rand(t, d) + 12 * w[y].float()).to(w.dtype)
    lse = bk.linear_cross_entropy(h, w, y)[1].double()
    want = torch.logsumexp(h.double() @ w.double().t(), 1)
    assert float((lse - want).norm() / want.norm()) <= 2 * 512 / 16 * 2.0 ** -26 + 2.0 ** -22
