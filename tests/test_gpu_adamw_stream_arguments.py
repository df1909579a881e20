"""AdamW on another stream (stream=) checks its arguments as on the current one, and takes lists of any kind."""

import pytest

from test_gpu_int8_matmul import bk  # noqa: F401

pytestmark = pytest.mark.gpu


def test_refusals(bk):  # noqa: F811
    import torch

    side = torch.cuda.Stream()
    p, g = [torch.ones(300, device="cuda")], [torch.ones(300, device="cuda")]
    s = bk.adamw_states(p)
    for call in (lambda **k: bk.adamw([p[0].cpu()], g, s, 1, **k), lambda **k: bk.adamw(p, [g[0].cpu()], s, 1, **k),
                 lambda **k: bk.adamw(p, [None], s, 1, **k), lambda **k: bk.adamw(p, [1.0], s, 1, **k),
                 lambda **k: bk.adamw(p, g, {**s, "m": [s["m"][0].cpu()]}, 1, **k),
                 lambda **k: bk.adamw(p, g, s, 1, copies=[p[0].cpu().half()], **k),
                 lambda **k: bk.adamw(p, g, s, torch.tensor(1), **k), lambda **k: bk.adamw(p, g, s, 1, skip=torch.tensor(1), **k)):
        for stream in (None, side):
            with pytest.raises(ValueError):
                call(stream=stream)
    torch.cuda.synchronize()
    assert bool((p[0] == 1).all())


@pytest.mark.parametrize("kind", [list, tuple, iter])
def test_lists_of_any_kind(bk, kind):  # noqa: F811
    import torch

    out = []
    for stream in (None, torch.cuda.Stream()):
        p = [torch.arange(300.0, device="cuda"), torch.ones(7, device="cuda")]
        g, copies = [torch.ones_like(t) for t in p], [torch.empty(300, dtype=torch.float16, device="cuda"), None]
        s = bk.adamw_states(p)
        torch.cuda.synchronize()
        bk.adamw(kind(p), kind(g), {k: kind(l) for k, l in s.items()}, 1, copies=kind(copies), stream=stream)
        torch.cuda.synchronize()
        out.append([*p, *s["m"], *s["v"], copies[0]])
    assert all(torch.equal(a, b) for a, b in zip(*out)) and not torch.equal(out[0][0], torch.arange(300.0, device="cuda"))
