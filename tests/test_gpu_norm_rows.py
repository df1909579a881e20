"""The norms and their gradients where a block (or a cluster of them) walks over many rows: rows fetched ahead, exchange
buffers taken in turns, gates that change within a range, several groups in a range, results in the inputs' place.
Tolerances: those of test_gpu_norm_residual.py, whose derivation counts a row's sums and, over tokens, their number."""

import pytest

from test_gpu_norm_residual import ALPHA, C, EPS, _forward, _make, _reference_gradients, _within, bk  # noqa: F401

pytestmark = pytest.mark.gpu

# Blocks of 512 threads: two for each of 152 SMs; of 1024, one; narrow rows: up to 32 of one warp.
FORWARD = [(1500, 4096, 1), (1500, 4096, 5), (1501, 4095, 19), (700, 9000, 7), (701, 9001, 1), (400, 20000, 8), (401, 32765, 1),
           (12000, 72, 6000), (20000, 40, 1), (15001, 33, 7)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("t,d,groups", FORWARD)
def test_forward_over_many_rows(bk, t, d, groups, dtype, kind):  # noqa: F811
    import torch

    t = t // groups * groups
    x, h, _, _, a = _make(t, d, dtype, kind, groups)
    y, z = bk.norm_residual(x, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
    y2, c, s = bk.norm_residual(x, h, **a, alpha=ALPHA, eps=EPS, kind=kind, codes=True)
    assert torch.equal(y, y2)
    ry, ym, rz, zm = _forward(x, h, a, kind)
    _within(y, ry, ym, dtype)
    _within(z, rz, zm, dtype)
    s = s.double()[:, None]
    top = rz.abs().amax(1, keepdim=True)
    assert bool(((s * 127 - top).abs() <= (C * zm).amax(1, keepdim=True) + 2.0 ** -23 * top).all())
    assert bool(((c.double() * s - rz).abs() <= 0.5 * s * (1 + 1e-4) + C * zm).all())


# Up to 4096 columns in registers (32-bit elements through two stages of shared memory), wider rows in shared memory and
# clusters of up to eight blocks.  Groups: none, one, some that share ranges, and more of them than ranges (4000 x 72: 1216).
BACKWARD = [(1500, 4096, 0), (1500, 4096, 1), (1500, 4096, 5), (1501, 4095, 1), (2000, 1000, 1000), (3333, 515, 11), (900, 14336, 0),
            (900, 14336, 5), (901, 9001, 17), (600, 32768, 1), (300, 20000, 300), (4000, 72, 2000), (4000, 72, 4000), (7001, 33, 1)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("t,d,groups", BACKWARD)
def test_backward_over_many_rows(bk, t, d, groups, dtype, kind):  # noqa: F811
    t = t // max(1, groups) * max(1, groups)
    y, h, dy, dz, a = _make(t, d, dtype, kind, groups)
    got = bk.norm_residual_backward(dy, dz, y, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
    ref = _reference_gradients(dy, dz, y, h, a, kind)
    for name, value in got.items():
        if kind == "rms" and name.endswith("bias") or (name == "gate" and not groups):
            assert value is None
            continue
        full = name in ("X", "H")
        _within(value, *ref[name], dtype if full else "float32", C if full else C + t * 2.0 ** -24)


def _entry(name, *args):
    import torch

    from kronecker_hessian_gptq_gb300 import _lib

    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    _lib.check(getattr(_lib.load(), name)(*args, torch.cuda.current_stream().cuda_stream), name)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("t,d", [(1200, 4096), (1201, 1999), (700, 9000), (500, 14335), (5000, 72)])
def test_results_in_the_place_of_inputs(bk, t, d, dtype, kind):  # noqa: F811
    """Y in X or in H; dX in dY or in dZ, dH in H: bit for bit what apart they are."""
    import torch

    code, layer = {"float32": 0, "bfloat16": 2}[dtype], int(kind == "layer")
    x, h, dy, dz, a = _make(t, d, dtype, kind, 1)
    y, z = bk.norm_residual(x, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
    for which in "xh":
        i = {"x": x.clone(), "h": h.clone()}
        z2 = torch.empty_like(z)
        _entry("bakron_norm_residual", i["x"], d, i["h"], d, a["post"], a["post_bias"], a["gate"], d, 1, a["pre"], a["pre_bias"],
               ALPHA, EPS, layer, code, t, d, i[which], z2, None, None)
        assert torch.equal(i[which], y) and torch.equal(z2, z)
    g = bk.norm_residual_backward(dy, dz, y, h, **a, alpha=ALPHA, eps=EPS, kind=kind)
    n = bk.load_library().bakron_norm_residual_backward_workspace_size(t, d, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for which in ("dy", "dz"):
        i = {"dy": dy.clone(), "dz": dz.clone(), "h": h.clone()}
        f = {k: None if v is None else torch.empty_like(v) for k, v in g.items() if k not in "XH"}
        _entry("bakron_norm_residual_backward", i["dy"], d, i["dz"], d, y, d, i["h"], d, a["post"], a["post_bias"], a["gate"], d, 1,
               a["pre"], ALPHA, EPS, layer, code, t, d, i[which], i["h"], f["post"], f["post_bias"], f["gate"], f["pre"],
               f["pre_bias"], ws, n)
        assert torch.equal(i[which], g["X"]) and torch.equal(i["h"], g["H"])
        assert all(f[k] is None or torch.equal(f[k], g[k]) for k in f)
