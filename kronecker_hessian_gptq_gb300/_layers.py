"""Bindings of the layer operators: the 8-bit product, the norms around a
block with its gate and residual sum, and the cross entropy over a large
vocabulary with its gradient.

Like the rest of the package these marshal torch tensors into the C ABI and
enqueue on the current stream.  With stream=s a call runs as under
``with torch.cuda.stream(s)``: results and workspace belong to s, and the
inputs are kept from reuse until s has passed the call.  Zero tokens are
allowed everywhere and launch nothing.  Like the rest of the package the calls
are not recorded by autograd: gradients come from the calls that return them.

A call for one token takes less time on the GPU than a handful of torch calls
take on the host, so the checks here read each attribute once.
"""

from __future__ import annotations

import torch

from . import _lib

_F32 = torch.float32
_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_I8 = 3
_KINDS = {"rms": 0, "layer": 1}
_empty = torch.empty
_current_device = torch.cuda.current_device
_entries = {}


def _entry(name):
    """The C entry point `name`, looked up once."""
    f = _entries.get(name)
    if f is None:
        f = _entries[name] = getattr(_lib.load(), name)
    return f


def _call(name, *args):
    st = _entry(name)(*args)
    if st:
        _lib.check(st, name)


def _handle(device):
    return torch.cuda.current_stream(device).cuda_stream


# The same without the Stream object around it, where torch offers it.
_handle = getattr(torch._C, "_cuda_getCurrentRawStream", _handle)


def _on(stream, call, *args, **kw):
    """`call` as under the stream, with its inputs kept until the stream has passed it."""
    for t in (*args, *kw.values()):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _names(dtypes):
    return " or ".join(str(d).replace("torch.", "") for d in dtypes)


def _matrix(t, name, dtypes):
    """Shape, row stride and device index of a 2-D CUDA tensor with contiguous rows."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and t.dtype in dtypes):
        raise ValueError(f"{name} must be a 2-D {_names(dtypes)} CUDA tensor")
    rows, cols = t.shape
    ld, one = t.stride()
    if cols < 1:
        raise ValueError(f"{name} must have at least one column")
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:  # a lone row may carry any stride
        ld = cols
    elif ld < cols:
        raise ValueError(f"the rows of {name} must not overlap (an expanded tensor: make it contiguous)")
    return rows, cols, ld, t.get_device()


def _like(t, name, dtype, rows, cols, device):
    """Row stride of a matrix of the given type, shape and device."""
    r, c, ld, d = _matrix(t, name, (dtype,))
    if r != rows or c != cols or d != device:
        raise ValueError(f"{name} must be {rows} x {cols} on cuda:{device}")
    return ld


def _vector(t, name, dtype, n, device):
    """Address of a dense vector, or None."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 1 and t.shape[0] == n
            and t.get_device() == device and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {_names((dtype,))} CUDA tensor of shape ({n},) on cuda:{device}")
    return t.data_ptr()


def _stream_on(device):
    if device != _current_device():
        raise ValueError(f"the tensors are on cuda:{device}, which is not the current device")
    return _handle(device)


def quantize_tokens(X, stream=None):
    """8-bit codes of activations X (T x K fp32, fp16 or bf16) with one scale
    for each token, max |x| / 127 (bakron_quantize_tokens).  Returns (codes
    int8 T x K, scales float32 T)."""
    if stream is not None:
        return _on(stream, quantize_tokens, X)
    T, K, ld, device = _matrix(X, "X", _CODES)
    C = _empty((T, K), dtype=torch.int8, device=X.device)
    s = _empty(T, dtype=_F32, device=X.device)
    if T:
        _call("bakron_quantize_tokens", X.data_ptr(), _CODES[X.dtype], T, K, ld, C.data_ptr(), s.data_ptr(),
              _stream_on(device))
    return C, s


_VALUES_OR_CODES = (*_CODES, torch.int8)
_BYTES = (torch.int8, torch.uint8)


def int8_matmul(X, codes, scales, x_scales=None, bias=None, dtype=None, stream=None):
    """Y = X V^T for a layer of 8-bit codes (N x K, int8, or the uint8 of
    pack_codes(V, 8)) with one scale for each output (bakron_int8_matmul).

    X (T x K) holds values, quantized in the call with one scale for each
    token, or int8 codes with x_scales (quantize_tokens, norm_residual).
    dtype is Y's: X's own for values, float32 for codes.  Returns (Y, status
    int32[1])."""
    if stream is not None:
        return _on(stream, int8_matmul, X, codes, scales, x_scales, bias, dtype)
    T, K, ldx, device = _matrix(X, "X", _VALUES_OR_CODES)
    N, cols, ldc, where = _matrix(codes, "codes", _BYTES)
    if cols != K or where != device:
        raise ValueError(f"codes must have {K} columns, on cuda:{device}")
    if N < 1:
        raise ValueError("codes must have at least one row")
    at = X.device
    kind = _CODES.get(X.dtype, _I8)
    if kind == _I8:
        if x_scales is None:
            raise ValueError("x_scales are needed where X holds codes")
    elif x_scales is not None:
        raise ValueError("x_scales go with int8 codes; values are quantized in the call")
    if scales is None:
        raise ValueError("scales are needed")
    w, xs, b = (_vector(scales, "scales", _F32, N, device), _vector(x_scales, "x_scales", _F32, T, device),
                _vector(bias, "bias", _F32, N, device))
    if dtype is None:
        dtype = _F32 if kind == _I8 else X.dtype
    out = _CODES.get(dtype)
    if out is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    Y = _empty((T, N), dtype=dtype, device=at)
    status = _empty(1, dtype=torch.int32, device=at)
    if T == 0:
        return Y, status.zero_()
    p = codes.data_ptr()
    nbytes = _entry("bakron_int8_matmul_workspace_size")(T, K, N, 1 if p % 16 or ldc % 16 else 0)
    # Held until the call has returned: what is given back before the launches
    # may by then be another thread's.
    ws = _empty(nbytes, dtype=torch.uint8, device=at) if nbytes else None
    _call("bakron_int8_matmul", X.data_ptr(), kind, ldx, xs, p, ldc, w, b, T, K, N, Y.data_ptr(), out,
          ws.data_ptr() if nbytes else None, nbytes, status.data_ptr(), _stream_on(device))
    return Y, status


def _norm_arguments(T, D, H, like, device, post, gate, pre, post_bias, pre_bias, kind):
    """Checks what both directions take.  Returns H's stride, the addresses of
    post, post_bias, pre, pre_bias, the gate's address, stride and rows, and
    the kind's code."""
    layer = _KINDS.get(kind)
    if layer is None:
        raise ValueError("kind must be 'rms' or 'layer'")
    ldh = ldg = groups = 0
    g = None
    if H is None:
        if not (post is None and post_bias is None and gate is None):
            raise ValueError("post, post_bias and gate go with H")
    else:
        ldh = _like(H, "H", like.dtype, T, D, device)
    if post_bias is not None or pre_bias is not None:
        if not layer:
            raise ValueError("biases go with layer norms")
        if (post_bias is not None and post is None) or (pre_bias is not None and pre is None):
            raise ValueError("a bias goes with its norm's weight")
    if gate is not None:
        if gate.dim() == 1:
            gate = gate[None]
        groups = gate.shape[0]
        if groups < 1 or T % groups:
            raise ValueError(f"gate must have one row for each of equal groups of the {T} tokens")
        ldg = _like(gate, "gate", like.dtype, groups, D, device)
        g = gate.data_ptr()
    return (ldh, _vector(post, "post", _F32, D, device), _vector(post_bias, "post_bias", _F32, D, device),
            _vector(pre, "pre", _F32, D, device), _vector(pre_bias, "pre_bias", _F32, D, device), g, ldg, groups, layer)


def norm_residual(X, H, post=None, gate=None, pre=None, alpha=1.0, eps=1e-6, kind="rms", post_bias=None,
                  pre_bias=None, codes=False, stream=None):
    """Y = alpha X + gate * N(H; post, post_bias) and Z = N(Y; pre, pre_bias)
    in one pass (bakron_norm_residual): the norms after a block and before the
    next one, the block's gate and the residual sum.

    X, H: T x D (fp32, fp16 or bf16); H None: Y = alpha X.  post, pre and
    their biases: D, float32; a norm without weights is left out; biases go
    with layer norms.  gate: D, or groups x D with one row for each of equal
    groups of consecutive tokens, of X's type.  kind: "rms" or "layer".
    Returns (Y, Z), Z None without pre; with codes=True (Y, C, s) with Z as
    int8 codes and a scale for each token, for int8_matmul."""
    if stream is not None:
        return _on(stream, norm_residual, X, H, post, gate, pre, alpha, eps, kind, post_bias, pre_bias, codes)
    T, D, ldx, device = _matrix(X, "X", _CODES)
    if codes and pre is None:
        raise ValueError("codes are those of the norm's output: pre is needed")
    ldh, w, wb, v, vb, g, ldg, groups, layer = _norm_arguments(T, D, H, X, device, post, gate, pre, post_bias, pre_bias,
                                                               kind)
    dtype, at = X.dtype, X.device
    Y = _empty((T, D), dtype=dtype, device=at)
    Z = C = s = None
    if codes:
        C = _empty((T, D), dtype=torch.int8, device=at)
        s = _empty(T, dtype=_F32, device=at)
    elif pre is not None:
        Z = _empty((T, D), dtype=dtype, device=at)
    if T:
        _call("bakron_norm_residual", X.data_ptr(), ldx, None if H is None else H.data_ptr(), ldh, w, wb, g, ldg, groups,
              v, vb, alpha, eps, layer, _CODES[dtype], T, D, Y.data_ptr(), None if Z is None else Z.data_ptr(),
              None if C is None else C.data_ptr(), None if s is None else s.data_ptr(), _stream_on(device))
    return (Y, C, s) if codes else (Y, Z)


def norm_residual_backward(dY, dZ, Y, H, post=None, gate=None, pre=None, alpha=1.0, eps=1e-6, kind="rms",
                           post_bias=None, pre_bias=None, stream=None):
    """Gradients of norm_residual for the gradients dY, dZ of its results
    (either may be None), from its Y and H (bakron_norm_residual_backward).

    Returns a dict: "X", "H" of the inputs' type, and in float32 "post",
    "pre", "gate" (of the gate's shape) and, for layer norms, "post_bias",
    "pre_bias" (wherever their norms are there); None for what there is no
    gradient of."""
    if stream is not None:
        return _on(stream, norm_residual_backward, dY, dZ, Y, H, post, gate, pre, alpha, eps, kind, post_bias, pre_bias)
    T, D, ldy, device = _matrix(Y, "Y", _CODES)
    ldh, w, wb, v, _, g, ldg, groups, layer = _norm_arguments(T, D, H, Y, device, post, gate, pre, post_bias, pre_bias,
                                                              kind)
    if dY is None and dZ is None:
        raise ValueError("dY or dZ is needed")
    if dZ is not None and pre is None:
        raise ValueError("dZ goes with pre")
    dtype, at = Y.dtype, Y.device
    lddy = 0 if dY is None else _like(dY, "dY", dtype, T, D, device)
    lddz = 0 if dZ is None else _like(dZ, "dZ", dtype, T, D, device)
    make = lambda shape: _empty(shape, dtype=_F32, device=at)  # noqa: E731
    out = {"X": _empty((T, D), dtype=dtype, device=at),
           "H": None if H is None else _empty((T, D), dtype=dtype, device=at),
           "post": None if post is None else make(D),
           "pre": None if pre is None else make(D),
           "gate": None if gate is None else make(gate.shape),
           "post_bias": make(D) if layer and post is not None else None,
           "pre_bias": make(D) if layer and pre is not None else None}
    if T == 0:
        for t in out.values():
            if t is not None:
                t.zero_()
        return out
    nbytes = _entry("bakron_norm_residual_backward_workspace_size")(T, D, groups)
    ws = _empty(nbytes, dtype=torch.uint8, device=at)
    to = {k: None if t is None else t.data_ptr() for k, t in out.items()}
    _call("bakron_norm_residual_backward", None if dY is None else dY.data_ptr(), lddy,
          None if dZ is None else dZ.data_ptr(), lddz, Y.data_ptr(), ldy, None if H is None else H.data_ptr(), ldh, w, wb, g,
          ldg, groups, v, alpha, eps, layer, _CODES[dtype], T, D, to["X"], to["H"], to["post"], to["post_bias"], to["gate"],
          to["pre"], to["pre_bias"], ws.data_ptr(), nbytes, _stream_on(device))
    return out


_HALVES = (torch.float16, torch.bfloat16)


def _loss(name, H, W, targets, coef, grad):
    T, D, ldh, device = _matrix(H, "H", _HALVES)
    V, cols, ldw, where = _matrix(W, "W", (H.dtype,))
    if cols != D or where != device or V < 1:
        raise ValueError(f"W must have {D} columns and at least one row, on cuda:{device}")
    if targets is None:
        raise ValueError("targets are needed")
    y, c = _vector(targets, "targets", torch.int64, T, device), _vector(coef, "coef", _F32, T, device)
    dtype, at = H.dtype, H.device
    loss, lse = _empty(T, dtype=_F32, device=at), _empty(T, dtype=_F32, device=at)
    status = _empty(1, dtype=torch.int32, device=at)
    out = (_empty((T, D), dtype=dtype, device=at), _empty((V, D), dtype=dtype, device=at)) if grad else ()
    if T == 0:
        if grad:
            out[1].zero_()
        return (loss, lse, *out, status.zero_())
    h, w = H.data_ptr(), W.data_ptr()
    copies = 1 if h % 16 or w % 16 or ldh % 8 or ldw % 8 else 0  # some row does not start on 16 bytes
    nbytes = _entry("bakron_linear_cross_entropy_workspace_size")(T, D, V, grad, copies)
    ws = _empty(nbytes, dtype=torch.uint8, device=at)
    more = (c,) if grad else ()
    _call(name, h, ldh, w, ldw, _CODES[dtype], y, *more, T, D, V, loss.data_ptr(), lse.data_ptr(),
          *(t.data_ptr() for t in out), ws.data_ptr(), nbytes, status.data_ptr(), _stream_on(device))
    return (loss, lse, *out, status)


def linear_cross_entropy(H, W, targets, stream=None):
    """Softmax cross entropy of the logits H W^T, which are not kept
    (bakron_linear_cross_entropy): H (T x D) and W (V x D) in fp16 or bf16,
    targets int64 (negative: no target, loss 0).  Returns (loss float32 T,
    lse float32 T, status int32[1])."""
    if stream is not None:
        return _on(stream, linear_cross_entropy, H, W, targets)
    return _loss("bakron_linear_cross_entropy", H, W, targets, None, 0)


def linear_cross_entropy_grad(H, W, targets, coef=None, stream=None):
    """linear_cross_entropy with the gradients of sum_t coef[t] loss[t]
    (bakron_linear_cross_entropy_grad); coef float32 T, or None for the mean
    over the tokens with a target.  Returns (loss, lse, dH, dW, status), the
    gradients of the inputs' type."""
    if stream is not None:
        return _on(stream, linear_cross_entropy_grad, H, W, targets, coef)
    return _loss("bakron_linear_cross_entropy_grad", H, W, targets, coef, 1)
