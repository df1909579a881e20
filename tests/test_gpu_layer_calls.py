"""The layer operators as a program calls them: captured in a CUDA graph and replayed on other inputs, and from several
threads that share the default stream.  Results are equal bit for bit to calls by themselves."""

import threading

import pytest

from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu


def _calls(bk, t):  # noqa: F811
    """name -> (inputs that change from replay to replay, call of them)."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(t)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    d, n, v = 520, 700, 1003
    codes = torch.randint(-127, 128, (n, d), generator=gen, device="cuda").to(torch.int8)
    odd = torch.randint(-127, 128, (n, d + 1), generator=gen, device="cuda").to(torch.int8)[:, 1:]
    scales, post, pre, gate = torch.rand(n, generator=gen, device="cuda"), rand(d), rand(d), rand(1, d).bfloat16()
    head = (rand(v, d) * d ** -0.5).bfloat16()
    y = torch.randint(-3, v, (t,), generator=gen, device="cuda")
    x, h, dy, dz = (rand(t, d).bfloat16() for _ in range(4))
    norm = {"post": post, "gate": gate, "pre": pre}

    def chained(x, h):
        _, c, s = bk.norm_residual(x, h, **norm, codes=True)
        return bk.int8_matmul(c, codes, scales, x_scales=s, dtype=torch.bfloat16)

    return {
        "tokens": ([x], lambda x: bk.quantize_tokens(x)),
        "product": ([x], lambda x: bk.int8_matmul(x, codes, scales)),
        "product of rows off 16 bytes": ([x], lambda x: bk.int8_matmul(x, odd, scales)),
        "norm to product": ([x, h], chained),
        "norm": ([x, h], lambda x, h: bk.norm_residual(x, h, **norm)),
        "norm backward": ([dy, dz, x, h], lambda *a: tuple(g for g in bk.norm_residual_backward(*a, **norm).values() if g is not None)),
        "loss": ([h], lambda h: bk.linear_cross_entropy(h, head, y)),
        "loss gradient": ([h], lambda h: bk.linear_cross_entropy_grad(h, head, y)),
    }


NAMES = ["tokens", "product", "product of rows off 16 bytes", "norm to product", "norm", "norm backward", "loss", "loss gradient"]


@pytest.mark.parametrize("t", [1, 3, 70, 900])
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
            assert torch.equal(a, c) and torch.equal(b, c)


@pytest.mark.parametrize("name", NAMES)
def test_threads_that_share_a_stream(bk, name):  # noqa: F811
    """Each call keeps its own memory until all of it is enqueued, whoever else allocates meanwhile."""
    import torch

    shapes = [1, 40, 70, 333]
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
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
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
