"""The layer operators' entry points reject bad arguments on the host, before
anything is enqueued (no GPU: no call here gets as far as a launch)."""

import ctypes

import pytest

F32, F16, BF16, I8 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    import kronecker_hessian_gptq_gb300 as bk
    from kronecker_hessian_gptq_gb300 import build as b

    b.build()
    return bk.load_library()


def at(address):
    return ctypes.c_void_p(address)  # never dereferenced


def refused(call, good, code=1, /, **bad):
    """`call` with one argument after another of `good` replaced is refused with `code`."""
    for name, values in bad.items():
        assert name in good, name
        for v in values:
            args = {**good, name: v}
            assert call(*args.values()) == code, (name, v)


def test_quantize_tokens(lib):
    good = dict(X=at(0x1000), dtype=F32, T=2, K=8, ldx=8, codes=at(0x2000), scales=at(0x3000), stream=None)
    refused(lib.bakron_quantize_tokens, good, X=[None, at(0x1002)], dtype=[-1, I8, 7], T=[0, -1, 1 << 31], K=[0, 1 << 31],
            ldx=[7], codes=[None, at(0x1000)], scales=[None, at(0x3002)])


def test_int8_matmul(lib):
    size = lib.bakron_int8_matmul_workspace_size
    need, copies = size(40, 64, 16, 0), size(40, 64, 16, 1)
    assert 0 < need < copies
    for bad in ((0, 64, 16, 0), (40, 0, 16, 0), (40, 64, 0, 0), (40, 1 << 17, 16, 0)):
        assert size(*bad) == 0
    good = dict(X=at(0x1000), xt=BF16, ldx=64, xs=None, codes=at(0x2000), ldc=64, scales=at(0x3000), bias=None, T=40, K=64,
                N=16, Y=at(0x5000), yt=BF16, ws=at(0x100000), n=need, status=at(0x6000), stream=None)
    call = lib.bakron_int8_matmul
    refused(call, good, X=[None, at(0x1001)], xt=[I8, 9], ldx=[63], xs=[at(0x4000)], codes=[None], ldc=[63], scales=[None],
            T=[0], K=[0, 1 << 17], N=[0], Y=[None, at(0x5001), at(0x1000), at(0x2000)], yt=[I8, -1], status=[None])
    refused(call, good, 4, ws=[None, at(0x100010)], n=[need - 1])
    refused(call, {**good, "ldc": 65}, 4, n=[need, copies - 1])


def test_norm_residual(lib):
    p = {k: at(0x1000 * (i + 1)) for i, k in enumerate("XHYZCsgwb")}
    good = dict(X=p["X"], ldx=64, H=p["H"], ldh=64, post=p["w"], post_bias=None, gate=p["g"], ldg=64, groups=2, pre=p["w"],
                pre_bias=None, alpha=1.0, eps=1e-6, kind=0, dtype=BF16, T=4, D=64, Y=p["Y"], Z=p["Z"], codes=None,
                code_scales=None, stream=None)
    call = lib.bakron_norm_residual
    refused(call, good, X=[None, at(0x1001)], ldx=[63], H=[None, at(0x2001)], ldh=[63], post_bias=[p["b"]], groups=[0, 3],
            ldg=[63], pre=[None], pre_bias=[p["b"]], eps=[-1.0, float("nan")], kind=[2], dtype=[I8], T=[0, 1 << 31],
            D=[0, 32769], Y=[None, p["Z"], at(0x3001)], Z=[None, p["X"], p["H"]], codes=[p["C"]], code_scales=[p["s"]])
    refused(call, {**good, "kind": 1, "post": None, "pre_bias": None}, post_bias=[p["b"]])
    refused(call, {**good, "Z": None, "codes": p["C"], "code_scales": p["s"]}, code_scales=[None], codes=[p["X"], p["H"], p["Y"]])
    refused(call, {**good, "ldx": 80}, Y=[p["X"]])  # in place, but not where the rows are


def test_norm_residual_backward(lib):
    size = lib.bakron_norm_residual_backward_workspace_size
    need = size(4, 64, 2)
    assert need > 0 and size(0, 64, 2) == 0 and size(4, 0, 2) == 0 and size(4, 64, 3) == 0 and size(4, 32769, 2) == 0
    p = {k: at(0x1000 * (i + 1)) for i, k in enumerate(["dY", "dZ", "Y", "H", "w", "b", "g", "dX", "dH", "f1", "f2", "f3"])}
    good = dict(dY=p["dY"], lddy=64, dZ=p["dZ"], lddz=64, Y=p["Y"], ldy=64, H=p["H"], ldh=64, post=p["w"], post_bias=None,
                gate=p["g"], ldg=64, groups=2, pre=p["w"], alpha=1.0, eps=1e-6, kind=0, dtype=BF16, T=4, D=64, dX=p["dX"],
                dH=p["dH"], dpost=p["f1"], dpost_bias=None, dgate=p["f2"], dpre=p["f3"], dpre_bias=None, ws=at(0x100000),
                n=need, stream=None)
    call = lib.bakron_norm_residual_backward
    refused(call, good, dY=[at(0x1001)], lddy=[63], lddz=[63], Y=[None], ldy=[63], H=[None], ldh=[63], post=[None],
            post_bias=[p["b"]], gate=[None], ldg=[63], groups=[0, 3], pre=[None], eps=[-1.0], kind=[3], dtype=[I8], T=[0],
            D=[0, 32769], dX=[None, p["Y"], p["H"], p["g"], p["dH"]], dH=[None, p["dY"], p["dZ"], p["Y"]],
            dpost_bias=[p["b"]], dpre_bias=[p["b"]])
    refused(call, {**good, "dZ": None}, dY=[None])
    refused(call, good, 4, ws=[None, at(0x100010)], n=[need - 1])


def test_linear_cross_entropy(lib):
    size = lib.bakron_linear_cross_entropy_workspace_size
    assert size(0, 8, 8, 0, 0) == size(4, 0, 8, 0, 0) == size(4, 8, 0, 1, 0) == 0
    loss, grad = size(4, 64, 100, 0, 0), size(4, 64, 100, 1, 0)
    assert 0 < loss < grad < size(4, 64, 100, 1, 1)
    good = dict(H=at(0x1000), ldh=64, W=at(0x2000), ldw=64, dtype=BF16, y=at(0x3000), T=4, D=64, V=100, loss=at(0x4000),
                lse=at(0x5000), ws=at(0x100000), n=loss, status=at(0x6000), stream=None)
    bad = dict(H=[None, at(0x1001)], ldh=[63], W=[None, at(0x2001)], ldw=[63], dtype=[F32, I8], y=[None, at(0x3004)], T=[0],
               D=[0], V=[0], loss=[None], lse=[None, at(0x4000)], status=[None])
    refused(lib.bakron_linear_cross_entropy, good, **bad)
    refused(lib.bakron_linear_cross_entropy, {**good, "ldh": 65}, 4, n=[loss, size(4, 64, 100, 0, 1) - 1])  # copies
    refused(lib.bakron_linear_cross_entropy, good, 4, ws=[None, at(0x100010)], n=[loss - 1])
    good = {**{k: v for k, v in list(good.items())[:6]}, "coef": None, **{k: good[k] for k in ("T", "D", "V", "loss", "lse")},
            "dH": at(0x7000), "dW": at(0x8000), "ws": at(0x100000), "n": grad, "status": at(0x6000), "stream": None}
    refused(lib.bakron_linear_cross_entropy_grad, good, **bad, dH=[None, at(0x1000), at(0x2000), at(0x7001)],
            dW=[None, at(0x7000), at(0x1000), at(0x2000), at(0x8001)])
    refused(lib.bakron_linear_cross_entropy_grad, good, 4, ws=[None, at(0x100010)], n=[grad - 1])


def test_arrays_of_32_bits_off_their_elements(lib):
    """Weights, scales, gradients, losses and status words that do not start on 4 bytes."""
    off = at(0x9002)
    good = dict(X=at(0x1000), xt=I8, ldx=64, xs=at(0x4000), codes=at(0x2000), ldc=64, scales=at(0x3000), bias=None, T=40, K=64,
                N=16, Y=at(0x5000), yt=BF16, ws=at(0x100000), n=1 << 30, status=at(0x6000), stream=None)
    refused(lib.bakron_int8_matmul, good, xs=[off], scales=[off], bias=[off], status=[off])
    p = {k: at(0x1000 * (i + 1)) for i, k in enumerate("XHYZCsgwb")}
    good = dict(X=p["X"], ldx=64, H=p["H"], ldh=64, post=p["w"], post_bias=p["b"], gate=p["g"], ldg=64, groups=2, pre=p["w"],
                pre_bias=p["b"], alpha=1.0, eps=1e-6, kind=1, dtype=BF16, T=4, D=64, Y=p["Y"], Z=None, codes=p["C"],
                code_scales=p["s"], stream=None)
    refused(lib.bakron_norm_residual, good, post=[off], post_bias=[off], pre=[off], pre_bias=[off], code_scales=[off])
    p = {k: at(0x1000 * (i + 1)) for i, k in enumerate(["dY", "dZ", "Y", "H", "w", "b", "g", "dX", "dH", "f1", "f2", "f3", "f4", "f5"])}
    good = dict(dY=p["dY"], lddy=64, dZ=p["dZ"], lddz=64, Y=p["Y"], ldy=64, H=p["H"], ldh=64, post=p["w"], post_bias=p["b"],
                gate=p["g"], ldg=64, groups=2, pre=p["w"], alpha=1.0, eps=1e-6, kind=1, dtype=BF16, T=4, D=64, dX=p["dX"],
                dH=p["dH"], dpost=p["f1"], dpost_bias=p["f2"], dgate=p["f3"], dpre=p["f4"], dpre_bias=p["f5"],
                ws=at(0x100000), n=1 << 30, stream=None)
    refused(lib.bakron_norm_residual_backward, good, post=[off], post_bias=[off], pre=[off], dpost=[off], dpost_bias=[off],
            dgate=[off], dpre=[off], dpre_bias=[off])
    good = dict(H=at(0x1000), ldh=64, W=at(0x2000), ldw=64, dtype=BF16, y=at(0x3000), coef=at(0x3800), T=4, D=64, V=100,
                loss=at(0x4000), lse=at(0x5000), dH=at(0x7000), dW=at(0x8000), ws=at(0x100000), n=1 << 30, status=at(0x6000),
                stream=None)
    refused(lib.bakron_linear_cross_entropy_grad, good, coef=[off], loss=[off], lse=[off], status=[off])
    good = {k: v for k, v in good.items() if k not in ("coef", "dH", "dW")}
    refused(lib.bakron_linear_cross_entropy, good, loss=[off], lse=[off], status=[off])


def test_statistics_of_the_loss_are_bounded(lib):
    """8 bytes for 64 logits: taken in pieces of the tokens, of 256 MiB or 256 tokens, whatever the tokens' number."""
    size = lib.bakron_linear_cross_entropy_workspace_size
    for T, V in ((1 << 18, 1 << 17), (1 << 16, 1 << 24), ((1 << 31) - 1, 32000)):
        assert size(T, 64, V, 0, 0) <= max(1 << 28, 256 * V // 8) + 4 * T + 4096
