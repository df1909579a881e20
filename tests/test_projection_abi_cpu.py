"""The entry points of a projection in 8-bit floats (its product, the norms of
heads, the AdamW step) reject bad arguments on the host, before anything is
enqueued (no GPU: no call here gets as far as a launch)."""

import ctypes
import math

import pytest

from test_layers_abi_cpu import BF16, F32, I8, at, lib, refused  # noqa: F401

E4M3 = 4
NAN = float("nan")


def test_quantize_blocks(lib):  # noqa: F811
    good = dict(X=at(0x1000), dtype=F32, T=2, K=8, ldx=8, rows=1, cols=128, codes=at(0x2000), ldc=8, scales=at(0x3000), stream=None)
    refused(lib.bakron_quantize_blocks, good, X=[None, at(0x1002)], dtype=[-1, I8, E4M3], T=[0, -1, 1 << 31], K=[0, 1 << 31],
            ldx=[7], rows=[0, 2, 128 * 128], cols=[1, 64, 0], codes=[None, at(0x1000)], ldc=[7], scales=[None, at(0x3002)])


def test_fp8_matmul(lib):  # noqa: F811
    size = lib.bakron_fp8_matmul_workspace_size
    need, copies = size(40, 64, 16, BF16, 0), size(40, 64, 16, BF16, 1)
    assert 0 < need < copies
    for bad in ((0, 64, 16, F32, 0), (40, 0, 16, F32, 0), (40, 64, 0, F32, 0), (40, (1 << 20) + 1, 16, F32, 0),
                ((1 << 24) + 1, 64, 16, F32, 0), (40, 64, 16, I8, 0)):
        assert size(*bad) == 0
    good = dict(X=at(0x1000), xt=BF16, ldx=64, xs=None, codes=at(0x2000), ldc=64, scales=at(0x3000), bias=None, T=40, K=64,
                N=16, Y=at(0x5000), yt=BF16, ws=at(0x100000), n=need, status=at(0x6000), stream=None)
    call = lib.bakron_fp8_matmul
    refused(call, good, X=[None, at(0x1001)], xt=[I8, E4M3, 9], ldx=[63], xs=[at(0x4000)], codes=[None], ldc=[63],
            scales=[None, at(0x3001)], bias=[at(0x7002)], T=[0, (1 << 24) + 1], K=[0, (1 << 20) + 1], N=[0, (1 << 20) + 1],
            Y=[None, at(0x5001), at(0x1000), at(0x2000)], yt=[I8, E4M3, -1], status=[None, at(0x6002)])
    refused(call, good, 4, ws=[None, at(0x100010)], n=[need - 1])
    refused(call, {**good, "ldc": 65}, 4, n=[need, copies - 1])
    refused(call, {**good, "codes": at(0x2001)}, 4, n=[need, copies - 1])
    refused(call, {**good, "xt": E4M3, "xs": at(0x4000)}, xs=[None, at(0x4002)])


def test_fp8_matmul_backward(lib):  # noqa: F811
    size = lib.bakron_fp8_matmul_backward_workspace_size
    need, copies = size(40, 64, 16, 7, 0), size(40, 64, 16, 7, 1)
    assert 0 < size(40, 64, 16, 1, 0) < size(40, 64, 16, 3, 0) < need < copies
    assert size(0, 64, 16, 7, 0) == 0 and size(40, 1 << 21, 16, 7, 0) == 0
    good = dict(dY=at(0x1000), lddy=16, X=at(0x2000), ldx=64, dtype=BF16, codes=at(0x3000), ldc=64, scales=at(0x4000), T=40,
                K=64, N=16, dX=at(0x5000), dW=at(0x6000), dbias=at(0x7000), ws=at(0x100000), n=need, status=at(0x8000), stream=None)
    call = lib.bakron_fp8_matmul_backward
    refused(call, good, dY=[None, at(0x1001)], lddy=[15], X=[None, at(0x2001)], ldx=[63], dtype=[I8, E4M3], codes=[None], ldc=[63],
            scales=[None, at(0x4002)], T=[0], K=[0], N=[0], dX=[at(0x5001), at(0x6000), at(0x1000), at(0x2000), at(0x3000)],
            dW=[at(0x6001), at(0x1000), at(0x2000), at(0x3000)], dbias=[at(0x7001)], status=[None])
    refused(call, {**good, "dX": None}, dW=[None])
    refused(call, good, 4, ws=[None, at(0x100010)], n=[need - 1])
    refused(call, {**good, "ldc": 72}, 4, n=[need, copies - 1])


def _heads():
    return dict(Q=at(0x1000), qt=64, qh=16, Hq=4, K=at(0x2000), kt=32, kh=16, Hk=2, qw=at(0x3000), kw=at(0x3100), pos=at(0x4000),
                f=at(0x5000), R=16, pairs=0, eps=1e-6, dtype=BF16, T=3, D=16)


def test_head_norm_rotary(lib):  # noqa: F811
    good = {**_heads(), "YQ": at(0x6000), "YK": at(0x7000), "stream": None}
    refused(lib.bakron_head_norm_rotary, good, Q=[None, at(0x1001)], Hq=[-1, 65536], K=[None, at(0x2001)], Hk=[-1, 65536],
            qw=[at(0x3002)], kw=[at(0x3001)], pos=[None, at(0x4004)], f=[None, at(0x5004)], R=[-2, 15, 18], pairs=[-1, 2],
            eps=[-1.0, NAN], dtype=[I8, E4M3], T=[0, 1 << 31], D=[0, 1025],
            YQ=[None, at(0x6001), at(0x1000), at(0x2000), at(0x7000)], YK=[None, at(0x1000), at(0x2000)])
    refused(lib.bakron_head_norm_rotary, {**good, "Hk": 0}, Hq=[0])


def test_head_norm_rotary_backward(lib):  # noqa: F811
    size = lib.bakron_head_norm_rotary_backward_workspace_size
    need = size(3, 16)
    assert need > 0 and size(0, 16) == 0 and size(3, 0) == 0 and size(3, 1025) == 0 and size(1 << 31, 16) == 0
    good = {"dYQ": at(0x8000), "dqt": 64, "dqh": 16, "dYK": at(0x9000), "dkt": 32, "dkh": 16, **_heads(), "dQ": at(0xA000),
            "dK": at(0xB000), "dqw": at(0xC000), "dkw": at(0xD000), "ws": at(0x100000), "n": need, "stream": None}
    call = lib.bakron_head_norm_rotary_backward
    refused(call, good, dYQ=[None, at(0x8001)], dYK=[None], Q=[None, at(0x1001)], K=[None], Hq=[-1, 65536], qw=[None, at(0x3002)],
            kw=[None], pos=[None], f=[None], R=[15, 18], pairs=[2], eps=[NAN], dtype=[I8], T=[0], D=[0, 1025],
            dQ=[None, at(0xA001), at(0x8000), at(0x9000), at(0x1000), at(0x2000), at(0xB000)], dK=[None, at(0x9000), at(0x2000)],
            dqw=[at(0xC002)], dkw=[at(0xD001)])
    refused(call, good, 4, ws=[None, at(0x100010)], n=[need - 1])


class Tensor(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("param", "grad", "m", "v", "ms", "vs", "copy")] + [("n", ctypes.c_int64)] + \
               [(k, ctypes.c_int) for k in ("pt", "gt", "ct")]


def _adamw(lib, bits=8, tensor=None, **change):  # noqa: F811
    t = dict(param=0x1000, grad=0x2000, m=0x3000, v=0x4000, ms=0x5000, vs=0x6000, copy=0x7000, n=9, pt=F32, gt=BF16, ct=BF16)
    t.update(tensor or {})
    a = dict(tensors=ctypes.byref(Tensor(**t)), count=1, bits=bits, lr=1e-3, lr_dev=None, step=1, step_dev=None, b1=0.9, b2=0.99,
             eps=1e-8, wd=0.1, scale=1.0, scale_dev=None, skip=None, seed=0, ws=at(0x100000), n=lib.bakron_adamw_workspace_size(),
             status=at(0x8000), stream=None)
    a.update(change)
    return lib.bakron_adamw(*a.values())


def test_adamw(lib):  # noqa: F811
    from kronecker_hessian_gptq_gb300 import _projection

    assert ctypes.sizeof(Tensor) == _projection._TENSOR.size
    need = lib.bakron_adamw_workspace_size()
    for name, values in dict(tensors=[None], count=[-1], bits=[0, 16], lr=[NAN], lr_dev=[at(0x8002)], step=[0, -1], step_dev=[at(0x8004)],
                             b1=[1.0, -0.1, NAN], b2=[1.0, -0.1, NAN], eps=[-1.0, NAN], wd=[NAN], scale=[NAN], scale_dev=[at(0x8001)],
                             skip=[at(0x8002)], status=[None, at(0x8001)]).items():
        for v in values:
            assert _adamw(lib, **{name: v}) == 1, (name, v)
    for name, values in dict(param=[None, 0x1002, 0x2000, 0x3000, 0x4000, 0x7000], grad=[None, 0x2001, 0x3000, 0x4000],
                             m=[None, 0x4000], v=[None], ms=[None, 0x5002], vs=[None, 0x6001], copy=[0x7001], n=[-1], pt=[I8, E4M3],
                             gt=[I8, 9], ct=[F32, I8]).items():
        for v in values:
            assert _adamw(lib, tensor={name: v}) == 1, (name, v)
    assert _adamw(lib, 32, {"m": 0x3002}) == 1 and _adamw(lib, 32, {"v": 0x4001}) == 1
    for change in ({"ws": None}, {"ws": at(0x100010)}, {"n": need - 1}):
        assert _adamw(lib, **change) == 4
    assert math.isfinite(need)
