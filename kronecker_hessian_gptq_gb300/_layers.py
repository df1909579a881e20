"""Bindings of the layer operators: the 8-bit product, the norms around a
block with its gate and residual sum, and the cross entropy over a large
vocabulary with its gradient.

Like the rest of the package these marshal torch tensors into the C ABI and
enqueue on the current stream.  With stream=s a call runs as under
``with torch.cuda.stream(s)``: results and workspace belong to s, and the
inputs are kept from reuse until s has passed the call.  Zero tokens are
allowed everywhere and launch nothing.
"""

from __future__ import annotations

import functools

import torch

from . import _lib

_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_KINDS = {"rms": 0, "layer": 1}


def _on_stream(call):
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call(*args, **kw)

    return wrapped


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_of(t):
    device = t.device.index
    if device != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{device}, which is not the current device")
    return torch.cuda.current_stream(device).cuda_stream


def _require(t, name, dtypes, shape, device, dense=False):
    """A CUDA tensor of one of the types and of the shape, with contiguous rows."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.shape == shape and t.device == device):
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be a {kinds} CUDA tensor of shape {tuple(shape)} on {device}")
    if dense:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous rows")


def _matrix(t, name, dtypes):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 2 and t.dtype in dtypes):
        kinds = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be a 2-D {kinds} CUDA tensor")
    if t.shape[1] < 1:
        raise ValueError(f"{name} must have at least one column")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.shape


def _ld(t):
    """Row stride; a lone row (or column) may carry any, so the width stands in for it."""
    if t is None:
        return 0
    ld = t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else t.shape[-1]
    if ld < t.shape[-1]:
        raise ValueError("rows must not overlap (an expanded tensor: make it contiguous)")
    return ld


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


@_on_stream
def quantize_tokens(X):
    """8-bit codes of activations X (T x K fp32, fp16 or bf16) with one scale
    for each token, max |x| / 127 (bakron_quantize_tokens).  Returns (codes
    int8 T x K, scales float32 T)."""
    T, K = _matrix(X, "X", _CODES)
    C = torch.empty((T, K), dtype=torch.int8, device=X.device)
    s = torch.empty(T, dtype=torch.float32, device=X.device)
    if T:
        st = _lib.load().bakron_quantize_tokens(X.data_ptr(), _CODES[X.dtype], T, K, _ld(X), C.data_ptr(), s.data_ptr(),
                                                _stream_of(X))
        _lib.check(st, "bakron_quantize_tokens")
    return C, s


@_on_stream
def int8_matmul(X, codes, scales, x_scales=None, bias=None, dtype=None):
    """Y = X V^T for a layer of 8-bit codes (N x K, int8, or the uint8 of
    pack_codes(V, 8)) with one scale for each output (bakron_int8_matmul).

    X (T x K) holds values, quantized in the call with one scale for each
    token, or int8 codes with x_scales (quantize_tokens, norm_residual).
    dtype is Y's: X's own for values, float32 for codes.  Returns (Y, status
    int32[1])."""
    T, K = _matrix(X, "X", (torch.int8, *_CODES))
    N = _matrix(codes, "codes", (torch.int8, torch.uint8))[0]
    device, f32 = X.device, (torch.float32,)
    _require(codes, "codes", (codes.dtype,), (N, K), device)
    _require(scales, "scales", f32, (N,), device, dense=True)
    if X.dtype is torch.int8:
        if x_scales is None:
            raise ValueError("x_scales are needed where X holds codes")
        _require(x_scales, "x_scales", f32, (T,), device, dense=True)
    elif x_scales is not None:
        raise ValueError("x_scales go with int8 codes; values are quantized in the call")
    if bias is not None:
        _require(bias, "bias", f32, (N,), device, dense=True)
    if dtype is None:
        dtype = torch.float32 if X.dtype is torch.int8 else X.dtype
    if dtype not in _CODES:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    Y = torch.empty((T, N), dtype=dtype, device=device)
    status = torch.empty(1, dtype=torch.int32, device=device)
    if T == 0:
        return Y, status.zero_()
    lib = _lib.load()
    ws = _workspace(lib.bakron_int8_matmul_workspace_size(T, K, N, int(codes.data_ptr() % 16 + _ld(codes) % 16 > 0)), device)
    st = lib.bakron_int8_matmul(X.data_ptr(), _CODES.get(X.dtype, 3), _ld(X), _ptr(x_scales), codes.data_ptr(),
                                _ld(codes), scales.data_ptr(), _ptr(bias), T, K, N, Y.data_ptr(), _CODES[dtype],
                                _ptr(ws), 0 if ws is None else ws.numel(), status.data_ptr(), _stream_of(X))
    _lib.check(st, "bakron_int8_matmul")
    return Y, status


def _norm_arguments(T, D, H, like, post, gate, pre, post_bias, pre_bias, kind):
    """Checks what both directions take; returns (gate as groups x D, groups, kind's code)."""
    device, f32 = like.device, (torch.float32,)
    if kind not in _KINDS:
        raise ValueError("kind must be 'rms' or 'layer'")
    if H is None:
        if not (post is None and post_bias is None and gate is None):
            raise ValueError("post, post_bias and gate go with H")
    else:
        _require(H, "H", (like.dtype,), (T, D), device)
    for w, name in ((post, "post"), (post_bias, "post_bias"), (pre, "pre"), (pre_bias, "pre_bias")):
        if w is not None:
            _require(w, name, f32, (D,), device, dense=True)
    if (post_bias is not None and post is None) or (pre_bias is not None and pre is None):
        raise ValueError("a bias goes with its norm's weight")
    if kind == "rms" and not (post_bias is None and pre_bias is None):
        raise ValueError("biases go with layer norms")
    if gate is None:
        return None, 0, _KINDS[kind]
    if gate.dim() == 1:
        gate = gate[None]
    groups = gate.shape[0]
    _require(gate, "gate", (like.dtype,), (groups, D), device)
    if groups < 1 or T % groups:
        raise ValueError(f"gate must have one row for each of equal groups of the {T} tokens")
    return gate, groups, _KINDS[kind]


@_on_stream
def norm_residual(X, H, post=None, gate=None, pre=None, alpha=1.0, eps=1e-6, kind="rms", post_bias=None,
                  pre_bias=None, codes=False):
    """Y = alpha X + gate * N(H; post, post_bias) and Z = N(Y; pre, pre_bias)
    in one pass (bakron_norm_residual): the norms after a block and before the
    next one, the block's gate and the residual sum.

    X, H: T x D (fp32, fp16 or bf16); H None: Y = alpha X.  post, pre and
    their biases: D, float32; a norm without weights is left out; biases go with layer norms.  gate: D,
    or groups x D with one row for each of equal groups of consecutive tokens,
    of X's type.  kind: "rms" or "layer".  Returns (Y, Z), Z None without
    pre; with codes=True (Y, C, s) with Z as int8 codes and a scale for each
    token, for int8_matmul."""
    T, D = _matrix(X, "X", _CODES)
    if codes and pre is None:
        raise ValueError("codes are those of the norm's output: pre is needed")
    gate, groups, layer = _norm_arguments(T, D, H, X, post, gate, pre, post_bias, pre_bias, kind)
    Y = torch.empty((T, D), dtype=X.dtype, device=X.device)
    Z = torch.empty_like(Y) if pre is not None and not codes else None
    C = s = None
    if codes:
        C = torch.empty((T, D), dtype=torch.int8, device=X.device)
        s = torch.empty(T, dtype=torch.float32, device=X.device)
    if T:
        st = _lib.load().bakron_norm_residual(
            X.data_ptr(), _ld(X), _ptr(H), _ld(H), _ptr(post), _ptr(post_bias), _ptr(gate), _ld(gate), groups, _ptr(pre),
            _ptr(pre_bias), alpha, eps, layer, _CODES[X.dtype], T, D, Y.data_ptr(), _ptr(Z), _ptr(C), _ptr(s),
            _stream_of(X))
        _lib.check(st, "bakron_norm_residual")
    return (Y, C, s) if codes else (Y, Z)


@_on_stream
def norm_residual_backward(dY, dZ, Y, H, post=None, gate=None, pre=None, alpha=1.0, eps=1e-6, kind="rms",
                           post_bias=None, pre_bias=None):
    """Gradients of norm_residual for the gradients dY, dZ of its results
    (either may be None), from its Y and H (bakron_norm_residual_backward).

    Returns a dict: "X", "H" of the inputs' type, and in float32 "post",
    "pre", "gate" (of the gate's shape) and, for layer norms, "post_bias",
    "pre_bias" (wherever their norms are there); None for what there is no
    gradient of."""
    T, D = _matrix(Y, "Y", _CODES)
    shape = None if gate is None else gate.shape
    gate, groups, layer = _norm_arguments(T, D, H, Y, post, gate, pre, post_bias, pre_bias, kind)
    if dY is None and dZ is None:
        raise ValueError("dY or dZ is needed")
    if dZ is not None and pre is None:
        raise ValueError("dZ goes with pre")
    for t, name in ((dY, "dY"), (dZ, "dZ")):
        if t is not None:
            _require(t, name, (Y.dtype,), (T, D), Y.device)
    make = lambda *s: torch.empty(s, dtype=torch.float32, device=Y.device)  # noqa: E731
    out = {"X": torch.empty((T, D), dtype=Y.dtype, device=Y.device),
           "H": None if H is None else torch.empty((T, D), dtype=Y.dtype, device=Y.device),
           "post": None if post is None else make(D),
           "pre": None if pre is None else make(D),
           "gate": None if gate is None else make(*shape),
           "post_bias": make(D) if layer and post is not None else None,
           "pre_bias": make(D) if layer and pre is not None else None}
    if T == 0:
        for t in out.values():
            if t is not None:
                t.zero_()
        return out
    lib = _lib.load()
    ws = _workspace(lib.bakron_norm_residual_backward_workspace_size(T, D, groups), Y.device)
    st = lib.bakron_norm_residual_backward(
        _ptr(dY), _ld(dY), _ptr(dZ), _ld(dZ), Y.data_ptr(), _ld(Y), _ptr(H), _ld(H), _ptr(post), _ptr(post_bias),
        _ptr(gate), _ld(gate), groups, _ptr(pre), alpha, eps, layer, _CODES[Y.dtype], T, D, out["X"].data_ptr(),
        _ptr(out["H"]), _ptr(out["post"]), _ptr(out["post_bias"]), _ptr(out["gate"]), _ptr(out["pre"]),
        _ptr(out["pre_bias"]), _ptr(ws), ws.numel(), _stream_of(Y))
    _lib.check(st, "bakron_norm_residual_backward")
    return out


def _copies(H, W):
    """Whether some row does not start on 16 bytes."""
    return int(any(t.data_ptr() % 16 or _ld(t) % 8 for t in (H, W)))


def _loss_arguments(H, W, targets):
    T, D = _matrix(H, "H", (torch.float16, torch.bfloat16))
    V = _matrix(W, "W", (H.dtype,))[0]
    if V < 1:
        raise ValueError("W must have at least one row")
    _require(W, "W", (H.dtype,), (V, D), H.device)
    _require(targets, "targets", (torch.int64,), (T,), H.device, dense=True)
    make = lambda: torch.empty(T, dtype=torch.float32, device=H.device)  # noqa: E731
    return T, D, V, make(), make(), torch.empty(1, dtype=torch.int32, device=H.device)


@_on_stream
def linear_cross_entropy(H, W, targets):
    """Softmax cross entropy of the logits H W^T, which are not kept
    (bakron_linear_cross_entropy): H (T x D) and W (V x D) in fp16 or bf16,
    targets int64 (negative: no target, loss 0).  Returns (loss float32 T,
    lse float32 T, status int32[1])."""
    T, D, V, loss, lse, status = _loss_arguments(H, W, targets)
    if T == 0:
        return loss, lse, status.zero_()
    lib = _lib.load()
    ws = _workspace(lib.bakron_linear_cross_entropy_workspace_size(T, D, V, 0, _copies(H, W)), H.device)
    st = lib.bakron_linear_cross_entropy(H.data_ptr(), _ld(H), W.data_ptr(), _ld(W), _CODES[H.dtype], targets.data_ptr(),
                                         T, D, V, loss.data_ptr(), lse.data_ptr(), _ptr(ws), ws.numel(),
                                         status.data_ptr(), _stream_of(H))
    _lib.check(st, "bakron_linear_cross_entropy")
    return loss, lse, status


@_on_stream
def linear_cross_entropy_grad(H, W, targets, coef=None):
    """linear_cross_entropy with the gradients of sum_t coef[t] loss[t]
    (bakron_linear_cross_entropy_grad); coef float32 T, or None for the mean
    over the tokens with a target.  Returns (loss, lse, dH, dW, status), the
    gradients of the inputs' type."""
    T, D, V, loss, lse, status = _loss_arguments(H, W, targets)
    if coef is not None:
        _require(coef, "coef", (torch.float32,), (T,), H.device, dense=True)
    dH = torch.empty((T, D), dtype=H.dtype, device=H.device)
    dW = torch.empty((V, D), dtype=H.dtype, device=H.device)
    if T == 0:
        return loss, lse, dH, dW.zero_(), status.zero_()
    lib = _lib.load()
    ws = _workspace(lib.bakron_linear_cross_entropy_workspace_size(T, D, V, 1, _copies(H, W)), H.device)
    st = lib.bakron_linear_cross_entropy_grad(H.data_ptr(), _ld(H), W.data_ptr(), _ld(W), _CODES[H.dtype],
                                              targets.data_ptr(), _ptr(coef), T, D, V, loss.data_ptr(), lse.data_ptr(),
                                              dH.data_ptr(), dW.data_ptr(), _ptr(ws), ws.numel(), status.data_ptr(),
                                              _stream_of(H))
    _lib.check(st, "bakron_linear_cross_entropy_grad")
    return loss, lse, dH, dW, status
