"""Bindings of the operators of a projection in 8-bit floats: the product of
e4m3 codes with a scale for each block of 128 and its gradients, the norms of
queries and keys for each head with the position rotation and their gradients,
and the AdamW step over many tensors.

In the manner of the layer operators (_layers.py): torch tensors are marshalled
into the C ABI, work is enqueued on the current stream (or stream=), no call is
recorded by autograd, and zero tokens are allowed everywhere.

The calls are made natively (csrc/marshal.cpp) where nothing is wrong with
their arguments; what is not handled there comes back as None and goes through
the checks here, which say what is wrong, and ctypes.  So does every call where
that module was not built for this torch and this Python.
"""

from __future__ import annotations

import ctypes
import struct
import warnings

import torch

from . import _lib
from ._layers import (_BYTES, _CODES, _F32, _call, _empty, _entry, _like, _matrix, _names, _on, _stream_on, _vector)

_E4M3 = torch.float8_e4m3fn
_E4M3_CODE = 4
_BLOCKS = ((1, 128), (128, 1), (128, 128))
_GROUP = 256  # values that share a scale in 8-bit optimizer states


_native = None


class _Through:
    """In place of the native module where there is none: handles no call, so that each goes through ctypes."""

    @staticmethod
    def adamw(*args):
        return None

    fp8_matmul = fp8_matmul_backward = head_norm_rotary = head_norm_rotary_backward = adamw


def _fast():
    global _native
    _native = _lib.load_marshal()
    if _native is None:
        warnings.warn("there is no _marshal.so for this torch and this Python: calls go through ctypes, which takes 15 us more "
                      "of the host for each (python -c 'import __graft_entry__ as g; g.build()' makes one)", RuntimeWarning,
                      stacklevel=3)
        _native = _Through
    return _native


def _ceil(a, b):
    return -(-a // b)


def _codes(rows, cols, device):
    """Room for e4m3 codes in rows that start on 16 bytes."""
    ld = _ceil(cols, 16) * 16
    t = _empty((rows, ld), dtype=_E4M3, device=device)
    return t if ld == cols else t[:, :cols]


def quantize_blocks(X, block=(1, 128), stream=None):
    """e4m3 codes of X (T x K fp32, fp16 or bf16) with one scale for each
    block: (1, 128) for tokens, (128, 128) for weights, (128, 1) for a sum over
    tokens (bakron_quantize_blocks).  Returns (codes float8_e4m3fn T x K, in
    rows that start on 16 bytes, scales float32 ceil(T / rows) x ceil(K / cols))."""
    if stream is not None:
        return _on(stream, quantize_blocks, X, block)
    T, K, ld, device = _matrix(X, "X", _CODES)
    rows, cols = block = tuple(block)
    if block not in _BLOCKS:
        raise ValueError("block must be (1, 128), (128, 1) or (128, 128)")
    C = _codes(T, K, X.device)
    s = _empty((_ceil(T, rows), _ceil(K, cols)), dtype=_F32, device=X.device)
    if T:
        _call("bakron_quantize_blocks", X.data_ptr(), _CODES[X.dtype], T, K, ld, rows, cols, C.data_ptr(), C.stride(0),
              s.data_ptr(), _stream_on(device))
    return C, s


def _scales(t, name, rows, cols, device):
    """Address of a dense matrix of scales."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _F32 and t.shape == (rows, cols) and t.get_device() == device
            and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of shape ({rows}, {cols}) on cuda:{device}")
    return t.data_ptr()


_VALUES_OR_CODES = (*_CODES, _E4M3)
_WEIGHTS = (_E4M3, *_BYTES)


def _weights(codes, scales, K, N, device):
    """Address and stride of the weights' codes, address of their scales, and their rows."""
    rows, cols, ld, where = _matrix(codes, "codes", _WEIGHTS)
    if cols != K or where != device or rows < 1 or (N is not None and rows != N):
        raise ValueError(f"codes must have {K} columns and {'at least one row' if N is None else f'{N} rows'}, on cuda:{device}")
    return codes.data_ptr(), ld, _scales(scales, "scales", _ceil(rows, 128), _ceil(K, 128), device), rows


def fp8_matmul(X, codes, scales, x_scales=None, bias=None, dtype=None, stream=None):
    """Y = X V^T for a layer of e4m3 codes (N x K) with one scale for each
    128 x 128 (bakron_fp8_matmul; quantize_blocks gives both).

    X (T x K) holds values, quantized in the call with a scale for each 128 of
    a token, or float8_e4m3fn codes with x_scales (T x ceil(K / 128)).  dtype
    is Y's: X's own for values, float32 for codes.  Returns (Y, status
    int32[1])."""
    if stream is not None:
        return _on(stream, fp8_matmul, X, codes, scales, x_scales, bias, dtype)
    done = (_native or _fast()).fp8_matmul(X, codes, scales, x_scales, bias, -1 if dtype is None else _CODES.get(dtype, 9))
    if done is not None:
        return done
    T, K, ldx, device = _matrix(X, "X", _VALUES_OR_CODES)
    at = X.device
    p, ldc, w, N = _weights(codes, scales, K, None, device)
    kind = _CODES.get(X.dtype, _E4M3_CODE)
    if kind == _E4M3_CODE:
        if x_scales is None:
            raise ValueError("x_scales are needed where X holds codes")
        xs = _scales(x_scales, "x_scales", T, _ceil(K, 128), device)
    elif x_scales is not None:
        raise ValueError("x_scales go with float8_e4m3fn codes; values are quantized in the call")
    else:
        xs = None
    b = _vector(bias, "bias", _F32, N, device)
    if dtype is None:
        dtype = _F32 if kind == _E4M3_CODE else X.dtype
    out = _CODES.get(dtype)
    if out is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    Y = _empty((T, N), dtype=dtype, device=at)
    status = _empty(1, dtype=torch.int32, device=at)
    if T == 0:
        return Y, status.zero_()
    nbytes = _entry("bakron_fp8_matmul_workspace_size")(T, K, N, kind, 1 if p % 16 or ldc % 16 else 0)
    ws = _empty(nbytes, dtype=torch.uint8, device=at) if nbytes else None
    _call("bakron_fp8_matmul", X.data_ptr(), kind, ldx, xs, p, ldc, w, b, T, K, N, Y.data_ptr(), out,
          ws.data_ptr() if nbytes else None, nbytes, status.data_ptr(), _stream_on(device))
    return Y, status


def fp8_matmul_backward(dY, X, codes, scales, bias=False, stream=None):
    """Gradients of fp8_matmul for the gradient dY (T x N) of its result
    (bakron_fp8_matmul_backward).

    X: the values that went in (T x K, of dY's type), or None for no "W".
    Returns (dict, status): "X" (T x K) and "W" (N x K, the gradient of the
    values that the codes stand for) of dY's type, "bias" (N, float32) with
    bias=True; None for what there is no gradient of."""
    if stream is not None:
        return _on(stream, fp8_matmul_backward, dY, X, codes, scales, bias)
    done = (_native or _fast()).fp8_matmul_backward(dY, X, codes, scales, bias)
    if done is not None:
        return done
    T, N, lddy, device = _matrix(dY, "dY", _CODES)
    at, dtype = dY.device, dY.dtype
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError("codes must be a 2-D tensor")
    K = codes.shape[1]
    p, ldc, w, _ = _weights(codes, scales, K, N, device)
    ldx = 0 if X is None else _like(X, "X", dtype, T, K, device)
    out = {"X": _empty((T, K), dtype=dtype, device=at),
           "W": None if X is None else _empty((N, K), dtype=dtype, device=at),
           "bias": _empty(N, dtype=_F32, device=at) if bias else None}
    status = _empty(1, dtype=torch.int32, device=at)
    if T == 0:
        for t in out.values():
            if t is not None:
                t.zero_()
        return out, status.zero_()
    want = 1 + (2 if X is not None else 0) + (4 if bias else 0)
    nbytes = _entry("bakron_fp8_matmul_backward_workspace_size")(T, K, N, want, 1 if p % 16 or ldc % 16 else 0)
    ws = _empty(nbytes, dtype=torch.uint8, device=at)
    to = {k: None if t is None else t.data_ptr() for k, t in out.items()}
    _call("bakron_fp8_matmul_backward", dY.data_ptr(), lddy, None if X is None else X.data_ptr(), ldx, _CODES[dtype], p, ldc,
          w, T, K, N, to["X"], to["W"], to["bias"], ws.data_ptr(), nbytes, status.data_ptr(), _stream_on(device))
    return out, status


_PAIRS = {"halves": 0, "neighbours": 1}


def _heads(t, name, dtypes, T, D, device):
    """Address, strides of tokens and heads, and heads of a T x heads x D tensor."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 3 and t.dtype in dtypes):
        raise ValueError(f"{name} must be a 3-D {_names(dtypes)} CUDA tensor")
    n, heads, d = t.shape
    token, head, one = t.stride()
    if n != T or d != D or t.get_device() != device or heads > 65535:
        raise ValueError(f"{name} must have {T} tokens and at most 65535 heads of {D}, on cuda:{device}")
    if one != 1 and d > 1 and n * heads:
        raise ValueError(f"the values of a head of {name} must be contiguous")
    # A lone token or head may carry any stride.
    return t.data_ptr(), token if n > 1 else 0, head if heads > 1 else 0, heads


def _rotation(positions, freqs, T, D, device):
    if positions is None and freqs is None:
        return None, None, 0
    if positions is None or freqs is None:
        raise ValueError("positions and freqs go together")
    R = 2 * freqs.shape[0] if isinstance(freqs, torch.Tensor) and freqs.dim() == 1 else D + 1
    if R > D:
        raise ValueError(f"freqs must be a vector of at most {D // 2} frequencies, one for each pair of a head's values")
    return (_vector(positions, "positions", torch.int64, T, device),
            _vector(freqs, "freqs", torch.float64, R // 2, device), R)


def _pairs(pairs):
    code = _PAIRS.get(pairs)
    if code is None:
        raise ValueError("pairs must be 'halves' or 'neighbours'")
    return code


def _shape_of_heads(Q):
    if not (isinstance(Q, torch.Tensor) and Q.is_cuda and Q.dim() == 3 and Q.dtype in _CODES):
        raise ValueError(f"Q must be a 3-D {_names(_CODES)} CUDA tensor")
    T, _, D = Q.shape
    if not 1 <= D <= 1024:
        raise ValueError("heads must have 1 to 1024 values")
    return T, D, Q.get_device()


def head_norm_rotary(Q, K, positions, freqs, q_weight=None, k_weight=None, eps=1e-6, pairs="halves", stream=None):
    """Queries Q (T x heads x D) and keys K (T x heads x D, or None) with the
    RMS norm of each head (where its weight is given) and the rotation of its
    first 2 len(freqs) values by the position, in one pass
    (bakron_head_norm_rotary).

    Q and K: fp32, fp16 or bf16, views into a common buffer or not.  positions:
    int64 T.  freqs: float64, radians for each position (base ** (-2 i / R)),
    or both None.  Weights: D, float32.  pairs: "halves" (i, i + R / 2) or
    "neighbours" (2 i, 2 i + 1).  Returns (YQ, YK), dense; YK None without K."""
    if stream is not None:
        return _on(stream, head_norm_rotary, Q, K, positions, freqs, q_weight, k_weight, eps, pairs)
    done = (_native or _fast()).head_norm_rotary(Q, K, positions, freqs, q_weight, k_weight, eps, _PAIRS.get(pairs))
    if done is not None:
        return done
    T, D, device = _shape_of_heads(Q)
    dtype, at = Q.dtype, Q.device
    q, qt, qh, hq = _heads(Q, "Q", (dtype,), T, D, device)
    k, kt, kh, hk = (None, 0, 0, 0) if K is None else _heads(K, "K", (dtype,), T, D, device)
    if K is None and k_weight is not None:
        raise ValueError("k_weight goes with K")
    w, v = _vector(q_weight, "q_weight", _F32, D, device), _vector(k_weight, "k_weight", _F32, D, device)
    p, f, R = _rotation(positions, freqs, T, D, device)
    code = _pairs(pairs)
    YQ = _empty((T, hq, D), dtype=dtype, device=at)
    YK = None if K is None else _empty((T, hk, D), dtype=dtype, device=at)
    if T and hq + hk:
        _call("bakron_head_norm_rotary", q, qt, qh, hq, k, kt, kh, hk, w, v, p, f, R, code, eps, _CODES[dtype], T, D,
              YQ.data_ptr(), None if K is None else YK.data_ptr(), _stream_on(device))
    return YQ, YK


def head_norm_rotary_backward(dYQ, dYK, Q, K, positions, freqs, q_weight=None, k_weight=None, eps=1e-6, pairs="halves",
                              stream=None):
    """Gradients of head_norm_rotary for the gradients dYQ, dYK of its results,
    from its Q and K (bakron_head_norm_rotary_backward).  Returns a dict: "Q",
    "K" of the inputs' type, "q_weight", "k_weight" in float32; None for what
    there is no gradient of."""
    if stream is not None:
        return _on(stream, head_norm_rotary_backward, dYQ, dYK, Q, K, positions, freqs, q_weight, k_weight, eps, pairs)
    done = (_native or _fast()).head_norm_rotary_backward(dYQ, dYK, Q, K, positions, freqs, q_weight, k_weight, eps, _PAIRS.get(pairs))
    if done is not None:
        return done
    T, D, device = _shape_of_heads(Q)
    dtype, at = Q.dtype, Q.device
    q, qt, qh, hq = _heads(Q, "Q", (dtype,), T, D, device)
    k, kt, kh, hk = (None, 0, 0, 0) if K is None else _heads(K, "K", (dtype,), T, D, device)
    dq, dqt, dqh, heads = _heads(dYQ, "dYQ", (dtype,), T, D, device)
    dk = None
    dkt = dkh = 0
    if heads != hq or (K is None) != (dYK is None):
        raise ValueError("dYQ and dYK must have the heads of Q and K")
    if K is None:
        if k_weight is not None:
            raise ValueError("k_weight goes with K")
    else:
        dk, dkt, dkh, heads = _heads(dYK, "dYK", (dtype,), T, D, device)
        if heads != hk:
            raise ValueError("dYQ and dYK must have the heads of Q and K")
    w, v = _vector(q_weight, "q_weight", _F32, D, device), _vector(k_weight, "k_weight", _F32, D, device)
    p, f, R = _rotation(positions, freqs, T, D, device)
    code = _pairs(pairs)
    out = {"Q": _empty((T, hq, D), dtype=dtype, device=at),
           "K": None if K is None else _empty((T, hk, D), dtype=dtype, device=at),
           "q_weight": None if w is None else _empty(D, dtype=_F32, device=at),
           "k_weight": None if v is None else _empty(D, dtype=_F32, device=at)}
    if T == 0 or hq + hk == 0:
        for t in out.values():
            if t is not None:
                t.zero_()
        return out
    nbytes = _entry("bakron_head_norm_rotary_backward_workspace_size")(T, D)
    ws = _empty(nbytes, dtype=torch.uint8, device=at)
    to = {n: None if t is None else t.data_ptr() for n, t in out.items()}
    _call("bakron_head_norm_rotary_backward", dq, dqt, dqh, dk, dkt, dkh, q, qt, qh, hq, k, kt, kh, hk, w, v, p, f, R, code,
          eps, _CODES[dtype], T, D, to["Q"], to["K"], to["q_weight"], to["k_weight"], ws.data_ptr(), nbytes,
          _stream_on(device))
    return out


def adamw_states(params, bits=32):
    """States for adamw() of these parameters, all zero: a dict of lists "m"
    and "v" of float32, or, with bits=8, of float8_e4m3fn codes (of m and of
    the root of v), and "m_scales" and "v_scales", float32, one for each 256
    values."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    params = list(params)
    if bits == 32:
        return {name: [torch.zeros(p.numel(), dtype=_F32, device=p.device) for p in params] for name in ("m", "v")}
    states = {name: [torch.zeros(p.numel(), dtype=torch.uint8, device=p.device).view(_E4M3) for p in params]
              for name in ("m", "v")}
    for name in ("m_scales", "v_scales"):
        states[name] = [torch.zeros(_ceil(p.numel(), _GROUP), dtype=_F32, device=p.device) for p in params]
    return states


# A C bakron_adamw_tensor: seven pointers, the length, three types.
_TENSOR = struct.Struct("=7Qq3i4x")


def _dense(t, name, i, dtypes, n, device):
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.numel() == n and t.get_device() == device
            and t.is_contiguous()):
        raise ValueError(f"{name}[{i}] must be a contiguous {_names(dtypes)} CUDA tensor of {n} values on cuda:{device}")
    return t.data_ptr()


def _number(x, name, dtype, device):
    """(number, address): one of them, for a Python number or a tensor of one value."""
    if not isinstance(x, torch.Tensor):
        return x, None
    if x.dtype is not dtype or x.numel() != 1 or x.get_device() != device:
        raise ValueError(f"{name} must be a number or a {_names((dtype,))} CUDA tensor of one value on cuda:{device}")
    return 1, x.data_ptr()


def _pack(packed, params, lists, eight, device):
    """The tensors' list for the C ABI, one attribute after another, with what is wrong with them."""
    for name, l in lists.items():
        if len(l) != len(params):
            raise ValueError(f"{name} must have {len(params)} tensors, as params")
    kinds = (_E4M3,) if eight else (_F32,)
    for i, p in enumerate(params):
        pp = _dense(p, "params", i, _CODES, p.numel() if isinstance(p, torch.Tensor) else 0, device)
        n = p.numel()
        g = lists["grads"][i]
        gp = _dense(g, "grads", i, _CODES, n, device)
        mp, vp = (_dense(lists[k][i], k, i, kinds, n, device) for k in "mv")
        ms = vs = cp = ct = 0
        if eight:
            ms, vs = (_dense(lists[k][i], k, i, (_F32,), _ceil(n, _GROUP), device) for k in ("m_scales", "v_scales"))
        c = lists["copies"][i] if "copies" in lists else None
        if c is not None:
            cp, ct = _dense(c, "copies", i, (torch.float16, torch.bfloat16), n, device), _CODES[c.dtype]
        _TENSOR.pack_into(packed, i * _TENSOR.size, pp, gp, mp, vp, ms, vs, cp, n, _CODES[p.dtype], _CODES[g.dtype], ct)


def adamw(params, grads, states, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=1.0,
          copies=None, skip=None, seed=0, stream=None):
    """One AdamW step over all of params, in place (bakron_adamw).

    params: fp32, fp16 or bf16 tensors, dense; grads: of the same sizes, each
    in fp32, fp16 or bf16; states: adamw_states(params, bits).  copies: None, or
    a list of fp16 or bf16 tensors (or None) that get the new parameters too.
    step (from 1 on), lr and grad_scale: numbers, or CUDA tensors of one value
    (int64, float32, float32), which a captured call reads when it is replayed.
    skip: int32 CUDA tensor of one value; if it is not 0 everything stays as it
    is.  seed: of the random rounding of 8-bit states.  Autograd sees parameters
    and copies change in place, as it does with an optimizer of torch: a graph
    that kept one of them refuses to go backward.  Returns status int32[1]:
    DEV_NONFINITE_GRAD where values with such gradients were left as they are."""
    params, grads = list(params), list(grads)
    lists = {"grads": grads, **{k: list(l) for k, l in states.items()}}
    if copies is not None:
        lists["copies"] = list(copies)
    if stream is not None:
        for t in (*params, *(t for l in lists.values() for t in l), step, lr, grad_scale, skip):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        states = {k: l for k, l in lists.items() if k in states}
        with torch.cuda.stream(stream):
            return adamw(params, grads, states, step, lr, betas, eps, weight_decay, grad_scale, lists.get("copies"), skip, seed)
    eight = "m_scales" in states
    done = (_native or _fast()).adamw(params, grads, lists["m"], lists["v"], lists.get("m_scales"), lists.get("v_scales"),
                                      lists.get("copies"), step, lr, betas[0], betas[1], eps, weight_decay, grad_scale, skip, seed)
    if done is not None:
        return done
    if not params or not isinstance(params[0], torch.Tensor) or not params[0].is_cuda:
        raise ValueError("params must be CUDA tensors, at least one")
    device, at = params[0].get_device(), params[0].device
    count = len(params)
    packed = ctypes.create_string_buffer(count * _TENSOR.size)
    _pack(packed, params, lists, eight, device)
    rate, rate_dev = _number(lr, "lr", _F32, device)
    number, step_dev = _number(step, "step", torch.int64, device)
    scale, scale_dev = _number(grad_scale, "grad_scale", _F32, device)
    if step_dev is None and number < 1:
        raise ValueError("step must be at least 1")
    stop = None if skip is None else _number(skip, "skip", torch.int32, device)[1]
    if skip is not None and stop is None:
        raise ValueError(f"skip must be an int32 CUDA tensor of one value on cuda:{device}")
    status = _empty(1, dtype=torch.int32, device=at)
    nbytes = _entry("bakron_adamw_workspace_size")()
    ws = _empty(nbytes, dtype=torch.uint8, device=at)
    _call("bakron_adamw", packed, count, 8 if eight else 32, rate, rate_dev, number,
          step_dev, betas[0], betas[1], eps, weight_decay, scale, scale_dev, stop, seed & 0xFFFFFFFFFFFFFFFF, ws.data_ptr(),
          nbytes, status.data_ptr(), _stream_on(device))
    # A graph that kept one of them from before must not go backward with other values.
    torch.autograd.graph.increment_version([t for t in (*params, *lists.get("copies", ())) if t is not None
                                            and not t.is_inference()])
    return status
