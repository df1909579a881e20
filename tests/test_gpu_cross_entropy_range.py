"""Cross entropy where logits are large, masked or decided, with few tokens' coefficients of another size, and in several
pieces, against fp64.

Most inputs here are made so that a logit is one exact product (of whole numbers and powers of two in a few columns): the tensor cores'
sums then have no error, and what is left is the operator's own.  Tolerances, for logits that are exact: a row's sum of
exponentials is good to 2^-13 (1024 additions along any path, an exponential to 2^-21), which moves lse and loss by as
much, besides 2^-22 of their and the logits' sizes.  An entry of G is within p (2^-12 + 2^-13 + 2^-22 max |x|) + 2^-31 of
its coefficient before it is rounded to 16 bits: a step of the kept logarithms, the sum's error, and the rounding of
lse to fp32, which for large logits is what p is known to."""

import pytest

from test_gpu_cross_entropy import U, _close, _make, _reference, bk  # noqa: F401

pytestmark = pytest.mark.gpu


def _exact(h, w, y, coef):
    """fp64 (loss, tolerance), (lse, tolerance), G and its error for exact logits."""
    import torch

    x = h.double() @ w.double().t()
    has = (y >= 0) & (y < len(w))
    at = y.clamp(0, len(w) - 1)[:, None]
    lse = torch.logsumexp(x, 1)
    size = torch.where(x > lse[:, None] - 100, x.abs(), 0.0).amax(1)  # of the logits that count
    right = x.gather(1, at)[:, 0]
    # log-sum of the others, so that a loss near zero keeps its digits
    rest = torch.logsumexp(x.scatter(1, at, -float("inf")), 1)
    loss = torch.where(has, torch.nn.functional.softplus(rest - right), 0.0)
    loss = torch.where(has & (rest == -float("inf")), 0.0, loss)
    tol = 2.0 ** -13 + 2.0 ** -22 * size
    p = torch.exp(x - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, at, has.double()[:, None])
    c = torch.where(has, coef.double(), 0.0)[:, None]
    return (loss, tol * torch.clamp(loss, max=1.0) + 2.0 ** -22 * loss + 1e-30), (lse, tol), c * (p - hot), \
        c.abs() * (p * (2.0 ** -12 + tol[:, None]) + 2.0 ** -31)


def _check(bk, h, w, y, coef=None, finite=True):
    """Both calls against fp64, gradients too."""
    import torch

    dtype = str(h.dtype).replace("torch.", "")
    has = (y >= 0) & (y < len(w))
    given = has.float() / has.sum().clamp(min=1) if coef is None else coef
    loss, lse, g, err = _exact(h, w, y, given)
    got = bk.linear_cross_entropy(h, w, y)
    assert int(got[2].item()) == 0
    _close(got[0], *loss)
    _close(got[1], *lse)
    l2, s2, dh, dw, st = bk.linear_cross_entropy_grad(h, w, y, coef=coef)
    assert int(st.item()) == 0
    _close(l2, *loss)
    _close(s2, *lse)
    if finite:
        e = err + U[dtype] * (g.abs() + err)
        for out, a, b, ea in ((dh, g, w.double(), e), (dw, g.t(), h.double(), e.t())):
            ref = a @ b
            tol = ea @ b.abs() + (2 * a.shape[1] + 16) * 2.0 ** -24 * ((a.abs() + ea) @ b.abs())
            _close(out, ref, tol + U[dtype] * (ref.abs() + tol) + (2.0 ** -24 if dtype == "float16" else 1e-38))
    return loss[0], dh, dw


def _one_column(t, d, v, dtype, sizes, seed=0):
    """Logits h[t, 0] w[v, 0] + h[t, 1] w[v, 1]: a whole number of up to 8 bits times one of up to 3, or the like."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.zeros((t, d), device="cuda")
    w = torch.zeros((v, d), device="cuda")
    pick = torch.tensor(sizes, device="cuda", dtype=torch.float32)
    h[:, 0] = pick[torch.randint(0, len(sizes), (t,), generator=gen, device="cuda")]
    w[:, 0] = 1
    w[:, 1] = torch.randint(-6, 7, (v,), generator=gen, device="cuda").float()
    h[:, 1] = 1
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    to = getattr(torch, dtype)
    return h.to(to), w.to(to), y


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("v", [300, 9000])
def test_large_logits_of_a_row(bk, v, sign, dtype):  # noqa: F811
    """A row's logits all near +-5000 to 30000: what counts are their differences, 0 to 12."""
    sizes = [sign * s for s in (5120, 5760, 6016, 7168, 8192, 9984, 11008, 14336, 16256, 20480, 23040, 26624, 30720)]
    h, w, y = _one_column(150, 24, v, dtype, sizes)
    _check(bk, h, w, y)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("v", [200, 9000])
def test_a_row_decided_by_one_large_logit(bk, v, dtype):  # noqa: F811
    """One word far above the rest of its row, at the sizes where a rounded maximum leaves a remainder: p = 1 there, for the
    target (no gradient left) or for another word (all of it)."""
    import torch

    t = 120
    h = torch.zeros((t, 16), device="cuda")
    h[:, 0] = 5700 + 128 * torch.arange(t, device="cuda")
    w = torch.zeros((v, 16), device="cuda")
    w[v // 3, 0] = 1
    y = torch.full((t,), v // 3, device="cuda")
    y[::2] = v - 1
    to = getattr(torch, dtype)
    _check(bk, h.to(to), w.to(to), y)
    _check(bk, -h.to(to), w.to(to), y)


@pytest.mark.parametrize("mask", [-1e4, -6e4, -1e9, -1e30, -3.3895e38, -float("inf")])
@pytest.mark.parametrize("v,masked", [(700, 200), (700, 640), (9000, 8000), (65, 1)])
def test_masked_words(bk, v, masked, mask):  # noqa: F811
    """A column of ones in H and a mask's value in W leave words out, here whole runs of 64 of them, with the other logits
    far below zero too (an all-masked run is then the largest number about if it is taken for zero)."""
    import torch

    for low in (0.0, -120.0, -1000.0):
        gen = torch.Generator(device="cuda").manual_seed(v + masked)
        h = torch.zeros((40, 32), device="cuda")
        w = torch.zeros((v, 32), device="cuda")
        h[:, 0] = 1
        h[:, 1] = torch.randint(-4, 5, (40,), generator=gen, device="cuda").float()
        w[:, 0] = low
        w[v - masked:, 0] = mask
        w[:v - masked, 1] = torch.randint(-2, 3, (v - masked,), generator=gen, device="cuda").float()
        y = torch.randint(0, v - masked, (40,), generator=gen, device="cuda")
        y[::7] = -100
        loss, dh, dw = _check(bk, h.bfloat16(), w.bfloat16(), y, finite=mask > -float("inf"))
        assert torch.isfinite(loss).all()
        assert not dw[v - masked:].any()  # no token's probability reaches them


def test_a_masked_target_and_a_row_without_words(bk):  # noqa: F811
    import torch

    inf = float("inf")
    h = torch.zeros((4, 16), device="cuda")
    h[:, 0] = 1
    w = torch.zeros((200, 16), device="cuda")
    w[100:, 0] = -inf
    y = torch.tensor([3, 150, -1, 199], device="cuda")
    loss, lse, _ = bk.linear_cross_entropy(h.bfloat16(), w.bfloat16(), y)
    want = torch.log(torch.tensor(100.0, device="cuda"))
    assert torch.isposinf(loss[[1, 3]]).all() and loss[2] == 0 and (loss[0] - want).abs() < 1e-4
    assert ((lse - want).abs() < 1e-4).all()
    w[:, 0] = -inf
    for target in (-1, 5):
        loss, lse, _ = bk.linear_cross_entropy(h.bfloat16(), w.bfloat16(), torch.full((4,), target, device="cuda"))
        assert torch.isneginf(lse).all() and (torch.isnan(loss).all() if target >= 0 else not loss.any())


def test_an_infinite_logit_of_the_target(bk):  # noqa: F811
    """lse - x is infinity less infinity, whether or not another word is infinite too."""
    import torch

    h = torch.zeros((3, 16), device="cuda")
    h[:, 0] = 1
    w = torch.zeros((200, 16), device="cuda")
    w[70, 0] = float("inf")
    for words in (1, 2):
        w[69 + words, 0] = float("inf")
        loss, lse, dh, _, _ = bk.linear_cross_entropy_grad(h.bfloat16(), w.bfloat16(), torch.tensor([70, 3, -1], device="cuda"))
        assert torch.isnan(loss[:2]).all() and torch.isnan(lse).all() and loss[2] == 0 and torch.isnan(dh[:2]).any(1).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("v", [1000, 8193, 32000])
@pytest.mark.parametrize("logit", [5.0, 15.0, 30.0])
def test_losses_of_confident_tokens(bk, logit, v, dtype):  # noqa: F811
    """4096 terms for each logit, the target's about `logit`.  A loss is never negative, and its error is that of the
    others' log-sum below the target's logit: the tensor cores' sums of 4096 terms come out up to 2^-16 (256 steps of
    16 terms, 2^-24 each) of their size too small, of the others' about 5, the target's own sum is good to 2^-18 of it
    (128 sums of 32 terms, their magnitudes several times the logit), and all of it counts with 1 - p."""
    import torch

    t, d = 64, 4096
    gen = torch.Generator(device="cuda").manual_seed(v)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    w = (rand(v, d) * d ** -0.5).to(getattr(torch, dtype))
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    h = (rand(t, d) + logit * w[y].float()).to(w.dtype)
    x = h.double() @ w.double().t()
    right = x.gather(1, y[:, None])[:, 0]
    rest = torch.logsumexp(x.scatter(1, y[:, None], -float("inf")), 1)
    want = torch.nn.functional.softplus(rest - right)
    tol = -torch.expm1(-want) * (2.0 ** -16 * 5 + 2.0 ** -18 * right.abs()) + 2.0 ** -21 * want
    for loss, lse in (bk.linear_cross_entropy(h, w, y)[:2], bk.linear_cross_entropy_grad(h, w, y)[:2]):
        assert bool((loss >= 0).all()), float(loss.min())
        _close(loss, want, tol)
        _close(lse, want + right, tol + 2.0 ** -18 * right.abs())


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("logit", [10.0, 40.0])
def test_gradients_of_confident_tokens(bk, logit, dtype):  # noqa: F811
    """dH of a token that is right: c (p_y - 1) w_y and the others' p w, both of them about 1 - p."""
    import torch

    t, d, v = 32, 64, 500
    gen = torch.Generator(device="cuda").manual_seed(3)
    h, w = torch.zeros((t, d), device="cuda"), torch.zeros((v, d), device="cuda")
    w[:, 0] = torch.randint(-3, 4, (v,), generator=gen, device="cuda").float()
    w[:, 1 + t:] = torch.randint(-8, 9, (v, d - 1 - t), generator=gen, device="cuda").float()
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    each = torch.arange(t, device="cuda")
    w[y, 1 + each] = 1  # a column for each token, which its target alone answers to
    h[:, 0] = 0.25
    h[each, 1 + each] = logit
    h, w = h.to(getattr(torch, dtype)), w.to(getattr(torch, dtype))
    coef = torch.exp(torch.full((t,), min(logit, 20.0), device="cuda"))  # so that fp16 results are not below their steps
    _check(bk, h, w, y, coef)
    _, _, dh, _, _ = bk.linear_cross_entropy_grad(h, w, y, coef=coef)
    x = h.double() @ w.double().t()
    x, right = x.scatter(1, y[:, None], -float("inf")), x.gather(1, y[:, None])
    q = torch.sigmoid(torch.logsumexp(x, 1, keepdim=True) - right)  # 1 - p
    part = (torch.softmax(x, 1) * q).scatter(1, y[:, None], -q) * coef.double()[:, None]
    ref = part @ w.double()
    # Relative to 1 - p: a kept logarithm's step (2^-12), the sum of exponentials (2^-13), 500 terms' sum (2^-14), G's and
    # the result's rounding.  No word lies below the kept range here; G in fp16 ends 2^-39 below the largest coefficient.
    floor = 2.0 ** -39 * float(coef.max()) if dtype == "float16" else 0.0
    tol = (part.abs() * (2.0 ** -10 + U[dtype]) + floor) @ w.double().abs()
    _close(dh, ref, tol + U[dtype] * ref.abs() + 2.0 ** -24)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_a_coefficient_that_is_not_finite_keeps_to_its_token(bk, dtype, bad):  # noqa: F811
    """G[t] = coef[t] (p - hot): only row t of dH is touched (dW is a sum over all rows)."""
    import torch

    h, w, y = _make(140, 64, 400, dtype)
    y[:5] = 7
    coef = torch.rand(140, device="cuda") + 0.5
    clean = bk.linear_cross_entropy_grad(h, w, y, coef=coef)
    coef[3] = bad
    loss, lse, dh, dw, st = bk.linear_cross_entropy_grad(h, w, y, coef=coef)
    rest = torch.arange(140, device="cuda") != 3
    assert int(st.item()) == 0 and torch.equal(loss, clean[0]) and torch.equal(lse, clean[1])
    assert not torch.isfinite(dh[3]).any() and torch.isfinite(dh[rest]).all()
    # the largest coefficient, by which all are divided, may have been the third
    assert torch.allclose(dh[rest].float(), clean[2][rest].float(), rtol=4 * U[dtype], atol=4 * U[dtype] * float(clean[2].abs().max()))
    assert not torch.isfinite(dw).all()
    zero = bk.linear_cross_entropy_grad(h, w, y, coef=torch.where(rest, 0.0, coef))
    assert not zero[2][rest].any() and not torch.isfinite(zero[2][3]).any()


def test_losses_of_more_tokens_than_one_piece_holds(bk):  # noqa: F811
    """The loss alone, over a vocabulary so large that its statistics are taken in pieces of the tokens."""
    import torch

    h, w, y = _make(2600, 16, 1000003, "bfloat16")
    y[2500] = 1000003
    loss, lse, st = bk.linear_cross_entropy(h, w, y)
    assert int(st.item()) == 8
    for lo, hi in ((0, 700), (1900, 2200), (2300, 2600)):
        part = bk.linear_cross_entropy(h[lo:hi], w, y[lo:hi])
        assert torch.equal(part[0], loss[lo:hi]) and torch.equal(part[1], lse[lo:hi])
    for q in (slice(0, 20), slice(2040, 2060), slice(2590, 2600)):
        r = _reference(h[q], w, y[q])
        _close(loss[q], *r["loss"])
        _close(lse[q], *r["lse"])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("ratio", [1e-2, 1e-4, 1e-6])
@pytest.mark.parametrize("v", [500, 40000])
def test_gradients_of_tokens_with_small_coefficients(bk, v, ratio, dtype):  # noqa: F811
    """Tokens whose coefficient is `ratio` of the largest, which is such that their dH is well above fp16's steps.  In
    units of its coefficient a G is within p (2^-12 + 2^-13) + 2^-31, and 2^-40 / ratio besides: half of fp16's smallest
    step where the largest coefficient stands for 2^15 (bf16 has no such step here).  Roundings of G do not agree over
    the words: their sum over v is within six times its root of squares (the kept logarithms' and the sum's own part is
    taken in full)."""
    import torch

    t, d = 64, 48
    h, w, y = _make(t, d, v, dtype)
    y = y.clamp(min=0)
    coef = torch.full((t,), 1e-2 / ratio, device="cuda")
    coef[1::2] = 1e-2
    dh = bk.linear_cross_entropy_grad(h, w, y, coef=coef)[2][1::2].double()
    r = _reference(h, w, y, coef)
    small = slice(1, None, 2)
    g, err = r["g"][small], r["gerr"][small]
    step = 1e-2 * 2.0 ** -40 / ratio if dtype == "float16" else 0.0
    wd = w.double()
    ref = g @ wd
    tol = err @ wd.abs() + 6 * (((U[dtype] * g.abs() + step) ** 2) @ wd ** 2).sqrt() + (2 * v + 16) * 2.0 ** -24 * (g.abs() @ wd.abs())
    _close(dh, ref, tol + U[dtype] * ref.abs() + 2.0 ** -25)
    assert float((dh - ref).norm()) <= 8 * U[dtype] * float(ref.norm())
