"""The seed of an AdamW step's random rounding has 64 bits, and each of them counts."""

import numpy as np
import pytest

from test_gpu_adamw import ARGS, _check, _copy, _make
from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu


def test_every_bit_of_the_seed_counts(bk):  # noqa: F811
    import torch

    params, grads, states = _make(np.random.default_rng(1), [20000], "float32", "bfloat16", 8)

    def codes(seed):
        mine = _copy(states)
        bk.adamw([params[0].clone()], grads, mine, seed=seed, **ARGS)
        return mine["m"][0].view(torch.uint8)

    seen = [codes(5)] + [codes(5 ^ (1 << b)) for b in range(64)]
    assert torch.equal(seen[0], codes(5)) and torch.equal(codes(-1), codes((1 << 64) - 1))
    # Cut at other random numbers, about a third of values comes out another way; of 20000 never fewer than a tenth
    for i, a in enumerate(seen):
        for b in seen[:i]:
            assert int((a != b).sum()) > 2000


def test_a_seed_s_tensors_are_not_another_seed_s(bk):  # noqa: F811
    """Two equal tensors in a list: the second one's codes are those of no seed nearby for the first."""
    import torch

    params, grads, states = _make(np.random.default_rng(2), [20000], "float32", "bfloat16", 8)

    def codes(seed):
        p, g = [params[0].clone() for _ in range(2)], [grads[0]] * 2
        mine = {k: [l[0].clone() for _ in range(2)] for k, l in states.items()}
        bk.adamw(p, g, mine, seed=seed, **ARGS)
        return [c.view(torch.uint8) for c in mine["m"]]

    second = codes(3)[1]
    assert all(not torch.equal(second, codes(3 + (h << 32))[0]) for h in range(4))


def test_small_seeds_are_what_they_were(bk):  # noqa: F811
    params, grads, states = _make(np.random.default_rng(3), [5000, 300], "float32", "bfloat16", 8)
    before, old = [p.clone() for p in params], _copy(states)
    bk.adamw(params, grads, states, seed=(1 << 32) - 1, **ARGS)
    _check(before, grads, old, params, states, None, ARGS, seed=(1 << 32) - 1)
