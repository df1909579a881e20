"""The operators of a projection in 8-bit floats as a program calls them: captured in a CUDA graph and replayed on other
inputs, from several threads that share the default stream, and together in the example that trains a projection.
Results are equal bit for bit to calls by themselves."""

import os
import sys
import threading

import pytest

from conftest import ROOT
from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu


def _calls(bk, t):  # noqa: F811
    """name -> (inputs that change from replay to replay, call of them)."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(t)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    hq, hk, d, k = 5, 2, 64, 520
    n = (hq + hk) * d
    V, s = bk.quantize_blocks(rand(n, k) * k ** -0.5, (128, 128))
    odd = torch.empty((n, k + 1), dtype=torch.uint8, device="cuda")[:, 1:].copy_(V.view(torch.uint8))
    x, dy = rand(t, k).bfloat16(), rand(t, n).bfloat16()
    pos, freqs = torch.arange(t, device="cuda"), 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    qw, kw = 1 + 0.1 * rand(d), 1 + 0.1 * rand(d)
    some = lambda g: tuple(v for v in g.values() if v is not None)  # noqa: E731

    def head(y, back=None):
        y = y.view(t, hq + hk, d)
        a = (y[:, :hq], y[:, hq:], pos, freqs, qw, kw)
        if back is None:
            return bk.head_norm_rotary(*a)
        back = back.view(t, hq + hk, d)
        return some(bk.head_norm_rotary_backward(back[:, :hq], back[:, hq:], *a))

    def given(x):
        c, xs = bk.quantize_blocks(x)
        return bk.fp8_matmul(c, V, s, x_scales=xs, dtype=torch.bfloat16)

    return {
        "blocks": ([x], lambda x: (*bk.quantize_blocks(x), *bk.quantize_blocks(x, (128, 1)), *bk.quantize_blocks(x, (128, 128)))),
        "product": ([x], lambda x: bk.fp8_matmul(x, V, s)),
        "product of given codes": ([x], given),
        "product of rows off 16 bytes": ([x], lambda x: bk.fp8_matmul(x, odd, s)),
        "gradients": ([dy, x], lambda dy, x: some(bk.fp8_matmul_backward(dy, x, V, s, bias=True)[0])),
        "gradient of the values alone": ([dy], lambda dy: some(bk.fp8_matmul_backward(dy, None, odd, s)[0])),
        "heads": ([dy], head),
        "heads' gradients": ([dy, x], lambda dy, x: head(bk.fp8_matmul(x, V, s)[0], dy)),
        "product to heads": ([x], lambda x: head(bk.fp8_matmul(x, V, s)[0])),
    }


NAMES = ["blocks", "product", "product of given codes", "product of rows off 16 bytes", "gradients",
         "gradient of the values alone", "heads", "heads' gradients", "product to heads"]


def _equal(a, b):
    import torch

    return torch.equal(a.view(torch.uint8), b.view(torch.uint8)) if a.element_size() == 1 else torch.equal(a, b)


@pytest.mark.parametrize("t", [1, 3, 70, 300, 1500])
@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(bk, name, t):  # noqa: F811
    import torch

    inputs, call = _calls(bk, t)[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*inputs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        # twice in a row: the second call's first kernel follows the first one's last
        first = call(*inputs)
        second = call(*inputs)
    for turn in range(3):
        for i in inputs:
            i.copy_(i.flip(0) * (0.5 + turn))
        graph.replay()
        alone = call(*inputs)
        torch.cuda.synchronize()
        for a, b, c in zip(first, second, alone):
            assert _equal(a, c) and _equal(b, c)


@pytest.mark.parametrize("name", NAMES)
def test_threads_that_share_a_stream(bk, name):  # noqa: F811
    """Each call keeps its own memory until all of it is enqueued, whoever else allocates meanwhile."""
    import torch

    shapes = [1, 40, 130, 333]
    work = [_calls(bk, t)[name] for t in shapes]
    want = [call(*inputs) for inputs, call in work]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(work))

    def run(i):
        inputs, call = work[i]
        try:
            start.wait(timeout=30)
            for _ in range(20):
                got = call(*inputs)
                noise = torch.full((1 << 16,), float("nan"), device="cuda")
                if not all(_equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(shapes[i])
                del noise
        except Exception as e:  # a thread's failure is the test's
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=120)
    assert not wrong and not any(th.is_alive() for th in threads)


def test_two_graphs_at_once(bk):  # noqa: F811
    """Two captured calls, each with its own workspace in its graph's memory, replayed on two streams."""
    import torch

    made = []
    for t in (130, 900):
        inputs, call = _calls(bk, t)["gradients"]
        want = call(*inputs)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = call(*inputs)
        made.append((graph, got, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, _, _, stream in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, want, _ in made:
        assert all(_equal(a, b) for a, b in zip(got, want))


@pytest.fixture(scope="module")
def example(bk):  # noqa: F811
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import trained_projection
    finally:
        sys.path.pop(0)
    return trained_projection


def test_the_example_runs(bk, example):  # noqa: F811
    import math

    import torch

    losses, params = example.main(tokens=700, width=320, queries=3, keys=1, head=64, steps=4)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)
    assert all(bool(torch.isfinite(p).all()) for p in params.values())


def test_the_example_repeats_itself(bk, example):  # noqa: F811
    import torch

    runs = [example.main(tokens=333, width=256, queries=2, keys=1, head=48, steps=3, seed=1) for _ in range(2)]
    assert runs[0][0] == runs[1][0]
    assert all(torch.equal(runs[0][1][n], runs[1][1][n]) for n in runs[0][1])


def test_the_example_s_gradients(bk, example):  # noqa: F811
    """Against autograd in fp64 through the same blocks' values.  What differs: the codes of x (half a step: 2^-4 of a
    value or 2^-10 of its block's scale), y and the heads' gradients in bf16, and the codes of the sums for W; so the
    gradient of W is compared along its own direction and in norm, where half steps of either sign average out: each
    operand's codes are off by at most 2^-4, 2^-4 / sqrt(3) in the mean square, two of them 2^-4 sqrt(2 / 3) = 0.051,
    and the results of x's codes enter q - q* at the same size."""
    import torch

    layer, x, target, params = example.make(600, 256, 3, 1, 64, 3, seed=2)
    loss, grads, status = example.gradients(layer, params, x, target)
    assert int(status.item()) == 0
    c, s = bk.quantize_blocks(params["W"], (128, 128))
    V = (c.double() * s.double().repeat_interleave(128, 0)[: len(c)].repeat_interleave(128, 1)[:, : c.shape[1]]).requires_grad_()
    cx, sx = bk.quantize_blocks(x)
    vx = cx.double() * sx.double().repeat_interleave(128, 1)[:, : cx.shape[1]]
    qw, kw = params["q"].double().requires_grad_(), params["k"].double().requires_grad_()
    y = (vx @ V.t()).view(len(x), 4, 64)
    angle = layer["positions"].double()[:, None, None] * layer["freqs"]
    total = 0
    for part, w, t in ((y[:, :3], qw, target[0]), (y[:, 3:], kw, target[1])):
        n = part * (part.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = n[..., :32], n[..., 32:]
        out = torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)
        total = total + (out - t.double()).pow(2).mean()
    total.backward()
    assert abs(float(loss) - float(total.detach())) <= 0.02 * float(total.detach())
    for got, ref in ((grads["W"], V.grad), (grads["q"], qw.grad), (grads["k"], kw.grad)):
        off = float((got.double() - ref).norm() / ref.norm())
        assert off <= 0.1, off
