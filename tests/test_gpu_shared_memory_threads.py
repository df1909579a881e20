"""Calls that take more shared memory than a launch may take by itself, at several sizes from several threads: none lowers
what another one needs."""

import threading

import pytest

from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu


def _at_once(work, times):
    import torch

    want = [call() for call in work]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(work))

    def run(call, want):
        try:
            start.wait(timeout=30)
            for _ in range(times):
                if not all(torch.equal(a, b) for a, b in zip(call(), want)):
                    wrong.append("results")
        except Exception as e:  # a thread's failure is the test's
            wrong.append(e)

    threads = [threading.Thread(target=run, args=w) for w in zip(work, want)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=120)
    assert not wrong and not any(th.is_alive() for th in threads)


@pytest.mark.parametrize("widths", [(2048, 4096, 1000, 3000), (4104, 6000, 8000, 9216)])
def test_norm_residual_backward(bk, widths):  # noqa: F811
    import torch

    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731

    def call(y, dy, w):
        g = bk.norm_residual_backward(dy, None, y, y, post=w)
        return [t for t in g.values() if t is not None]

    _at_once([lambda a=(rand(300, d), rand(300, d), rand(d)): call(*a) for d in widths], 60)


def test_row_scales(bk):  # noqa: F811
    import torch

    gen = torch.Generator("cuda").manual_seed(2)
    work = [torch.randn((8, n), generator=gen, device="cuda") for n in (13000, 20000, 32000, 48000)]
    _at_once([lambda w=w: (bk.row_scales(w, -4, 3, grid=4),) for w in work], 60)
