"""Gradients of wide heads from several threads: each call of the kernel for any sizes takes its own amount of shared
memory, mostly of more than the 48 KB that a launch may take by itself, and no call lowers what another one needs."""

import threading

import numpy as np
import pytest

from test_gpu_head_norm import _args, _inputs
from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu


def test_sizes_of_shared_memory_at_the_same_time(bk):  # noqa: F811
    import torch

    # heads, width, rotated values: 67, 68, 51, 52 and 44 KB
    sizes = [(4, 1000, 1000), (2, 1024, 1024), (8, 1000, 1000), (8, 1023, 1000), (16, 1022, 1000)]
    work = []
    for i, (h, d, r) in enumerate(sizes):
        rng = np.random.default_rng(i)
        q, _ = _inputs(rng, 2000, h, 1, d, "bfloat16")
        dy, _ = _inputs(rng, 2000, h, 1, d, "bfloat16")
        p, f, (w, _) = _args(rng, 2000, d, r)
        call = lambda a=(dy, None, q, None, p, f, w): bk.head_norm_rotary_backward(*a)  # noqa: E731
        work.append((call, call()))
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(work))

    def run(call, want):
        try:
            start.wait(timeout=30)
            for _ in range(60):
                got = call()
                if not (torch.equal(got["Q"], want["Q"]) and torch.equal(got["q_weight"], want["q_weight"])):
                    wrong.append("results")
        except Exception as e:  # a thread's failure is the test's
            wrong.append(e)

    threads = [threading.Thread(target=run, args=w) for w in work]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=120)
    assert not wrong and not any(th.is_alive() for th in threads)
