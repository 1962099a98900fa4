"""Python face of the training operators of the C ABI.

Layer norm, gated feed-forward, softmax cross entropy of a linear classifier
and the linear layer, each as a forward and a backward function (the linear
layer's forward pass is ``linear``).  Every computation runs in
libjepa_gb300.so; torch supplies device memory and streams.

Tensors are contiguous and on one CUDA device, which need not be the current
one.  Work is enqueued on ``stream``, or on that device's current stream; the
outputs and the workspace are allocated on the stream that uses them, so
calls on several streams, and captured graphs, never share one.  Gradients
not asked for (``needs``) are returned as None.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from ._lib import check, load
from .binding import DTYPE_CODE, _ptr

_CODE = {torch.float32: DTYPE_CODE["f32"], torch.float16: DTYPE_CODE["f16"], torch.bfloat16: DTYPE_CODE["bf16"]}
_ACT = {"silu": _lib.GATE_SILU, "gelu": _lib.GATE_GELU}


def _expect(name, t, shape, dtype, device):
    """t is None or a contiguous tensor of this shape, dtype and device."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _matrix(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, has shape {tuple(t.shape)}")
    return t.shape


def _code(name, dtype):
    if dtype not in _CODE:
        raise ValueError(f"{name} is {dtype}: float32, float16 or bfloat16")
    return _CODE[dtype]


class _Launch:
    """The device and stream of one call: current while it allocates and launches."""

    def __init__(self, t, stream):
        if t.device.type != "cuda":
            raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
        self.device = t.device
        if stream is not None and stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, tensors are on {t.device}")
        self.stream = stream

    def __enter__(self):
        self._dev = torch.cuda.device(self.device)
        self._dev.__enter__()
        self._ctx = torch.cuda.stream(self.stream) if self.stream is not None else None
        if self._ctx is not None:
            self._ctx.__enter__()
        self.handle = C.c_void_p(torch.cuda.current_stream().cuda_stream)
        return self

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        self._dev.__exit__(*exc)

    def empty(self, shape, dtype, wanted=True):
        return torch.empty(shape, dtype=dtype, device=self.device) if wanted else None

    def workspace(self, nbytes):
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device)


def layernorm_fwd(x, w, b, eps, out_dtype=None, stream=None):
    """(y, mean, rstd) of x [..., dim] over its last dimension; w, b float
    [dim].  y has out_dtype (default x's; another one needs float32 x), mean
    and rstd are float32 of x's leading shape."""
    lib = load()
    dim = x.shape[-1]
    out_dtype = out_dtype or x.dtype
    xc, yc = _code("x", x.dtype), _code("out_dtype", out_dtype)
    _expect("x", x, x.shape, x.dtype, x.device)
    _expect("w", w, (dim,), torch.float32, x.device)
    _expect("b", b, (dim,), torch.float32, x.device)
    rows = x.numel() // dim if dim else 0
    with _Launch(x, stream) as la:
        y = la.empty(x.shape, out_dtype)
        mean, rstd = la.empty(x.shape[:-1], torch.float32), la.empty(x.shape[:-1], torch.float32)
        check(lib.jepa_layernorm_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd), rows, dim, xc, yc,
                                     eps, la.handle))
    return y, mean, rstd


def layernorm_bwd(dy, x, w, mean, rstd, residual=None, needs=(True, True), stream=None):
    """(dx, dw, db) from dy (y's shape and dtype), x, w and the forward pass's
    mean and rstd.  residual: x's shape and dtype, added to dx.  needs: (dw,
    db)."""
    lib = load()
    dim = x.shape[-1]
    xc, yc = _code("x", x.dtype), _code("dy", dy.dtype)
    dev = x.device
    for name, t, shape, dt in (("x", x, x.shape, x.dtype), ("dy", dy, x.shape, dy.dtype),
                               ("w", w, (dim,), torch.float32), ("mean", mean, x.shape[:-1], torch.float32),
                               ("rstd", rstd, x.shape[:-1], torch.float32), ("residual", residual, x.shape, x.dtype)):
        _expect(name, t, shape, dt, dev)
    rows = x.numel() // dim if dim else 0
    with _Launch(x, stream) as la:
        dx = la.empty(x.shape, x.dtype)
        dw, db = la.empty((dim,), torch.float32, needs[0]), la.empty((dim,), torch.float32, needs[1])
        ws = la.workspace(lib.jepa_layernorm_bwd_workspace_bytes(rows, dim))
        check(lib.jepa_layernorm_bwd(_ptr(dy), _ptr(x), _ptr(w), _ptr(mean), _ptr(rstd), _ptr(residual), _ptr(dx),
                                     _ptr(dw), _ptr(db), rows, dim, xc, yc, _ptr(ws), ws.numel(), la.handle))
    return dx, dw, db


def _ce_args(x, W, bias, labels):
    M, D = _matrix("x", x)
    V = _matrix("W", W)[0]
    code = _code("x", x.dtype)
    for name, t, shape, dt in (("x", x, x.shape, x.dtype), ("W", W, (V, D), x.dtype),
                               ("bias", bias, (V,), torch.float32)):
        _expect(name, t, shape, dt, x.device)
    if labels.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"labels are {labels.dtype}: int64 or int32")
    _expect("labels", labels, (M,), labels.dtype, x.device)
    return M, D, V, code


def linear_ce_fwd(x, W, bias, labels, ignore_index=-100, smoothing=0.0, stream=None):
    """(loss, lse), float [M], of the classifier x W^T + bias: x [M, D], W
    [V, D] in one dtype, bias float [V] or None, labels int64 (or int32) [M].
    Rows with label ignore_index have loss 0."""
    lib = load()
    M, D, V, code = _ce_args(x, W, bias, labels)
    with _Launch(x, stream) as la:
        labels = labels.long()
        loss, lse = la.empty((M,), torch.float32), la.empty((M,), torch.float32)
        ws = la.workspace(lib.jepa_linear_ce_workspace_bytes(M, D, V, code, 0))
        check(lib.jepa_linear_ce_fwd(_ptr(x), _ptr(W), _ptr(bias), _ptr(labels), _ptr(loss), _ptr(lse), M, D, V, code,
                                     ignore_index, smoothing, _ptr(ws), ws.numel(), la.handle))
    return loss, lse


def linear_ce_bwd(dloss, x, W, bias, labels, lse, ignore_index=-100, smoothing=0.0, needs=(True, True, True),
                  stream=None):
    """(dx, dW, dbias) from dloss, the gradient of each row's loss (float [M],
    or one number for all rows: 1 / n for the mean of n rows), and the forward
    pass's lse.  needs: (dx, dW, dbias)."""
    lib = load()
    M, D, V, code = _ce_args(x, W, bias, labels)
    _expect("lse", lse, (M,), torch.float32, x.device)
    with _Launch(x, stream) as la:
        labels = labels.long()
        if not torch.is_tensor(dloss):
            dloss = torch.full((M,), float(dloss), device=x.device)
        elif dloss.dim() == 0:
            dloss = dloss.to(device=x.device, dtype=torch.float32).expand(M).contiguous()
        _expect("dloss", dloss, (M,), torch.float32, x.device)
        dx, dW = la.empty((M, D), x.dtype, needs[0]), la.empty((V, D), x.dtype, needs[1])
        dbias = la.empty((V,), torch.float32, needs[2])
        ws = la.workspace(lib.jepa_linear_ce_workspace_bytes(M, D, V, code, 1))
        check(lib.jepa_linear_ce_bwd(_ptr(x), _ptr(W), _ptr(bias), _ptr(labels), _ptr(lse), _ptr(dloss), _ptr(dx),
                                     _ptr(dW), _ptr(dbias), M, D, V, code, ignore_index, smoothing, _ptr(ws),
                                     ws.numel(), la.handle))
    return dx, dW, dbias


def _ffn_args(x, Wg, Wu, bg, bu, act):
    M, D = _matrix("x", x)
    F = _matrix("Wg", Wg)[0]
    code = _code("x", x.dtype)
    for name, t, shape, dt in (("x", x, x.shape, x.dtype), ("Wg", Wg, (F, D), x.dtype), ("Wu", Wu, (F, D), x.dtype),
                               ("bg", bg, (F,), torch.float32), ("bu", bu, (F,), torch.float32)):
        _expect(name, t, shape, dt, x.device)
    if act not in _ACT:
        raise ValueError(f"act {act!r}: 'silu' or 'gelu'")
    return M, D, F, code, _ACT[act]


def gated_ffn_fwd(x, Wg, Wu, bg=None, bu=None, act="silu", stream=None):
    """h = act(x Wg^T + bg) * (x Wu^T + bu), [M, F] in x's dtype: x [M, D],
    Wg, Wu [F, D]; bg, bu float [F] or None; act 'silu' or 'gelu' (erf)."""
    lib = load()
    M, D, F, code, a = _ffn_args(x, Wg, Wu, bg, bu, act)
    with _Launch(x, stream) as la:
        h = la.empty((M, F), x.dtype)
        ws = la.workspace(lib.jepa_gated_ffn_workspace_bytes(M, D, F, code, 0))
        check(lib.jepa_gated_ffn_fwd(_ptr(x), _ptr(Wg), _ptr(Wu), _ptr(bg), _ptr(bu), _ptr(h), M, D, F, code, a,
                                     _ptr(ws), ws.numel(), la.handle))
    return h


def gated_ffn_bwd(dh, x, Wg, Wu, bg=None, bu=None, act="silu", needs=(True, True, True, True, True), stream=None):
    """(dx, dWg, dWu, dbg, dbu) from dh [M, F]; the projections are computed
    again from x.  needs: one flag for each."""
    lib = load()
    M, D, F, code, a = _ffn_args(x, Wg, Wu, bg, bu, act)
    _expect("dh", dh, (M, F), x.dtype, x.device)
    with _Launch(x, stream) as la:
        dx = la.empty((M, D), x.dtype, needs[0])
        dWg, dWu = la.empty((F, D), x.dtype, needs[1]), la.empty((F, D), x.dtype, needs[2])
        dbg, dbu = la.empty((F,), torch.float32, needs[3]), la.empty((F,), torch.float32, needs[4])
        ws = la.workspace(lib.jepa_gated_ffn_workspace_bytes(M, D, F, code, 1))
        check(lib.jepa_gated_ffn_bwd(_ptr(dh), _ptr(x), _ptr(Wg), _ptr(Wu), _ptr(bg), _ptr(bu), _ptr(dx), _ptr(dWg),
                                     _ptr(dWu), _ptr(dbg), _ptr(dbu), M, D, F, code, a, _ptr(ws), ws.numel(),
                                     la.handle))
    return dx, dWg, dWu, dbg, dbu


def linear_bwd(dout, A, W, bias=True, needs=(True, True), stream=None):
    """(dA, dW, dbias) of out = A W^T + bias from dout [M, N]: A [M, K], W
    [N, K] and dout in one dtype.  needs: (dA, dW); bias: whether dbias (float
    [N]) is wanted."""
    lib = load()
    M, K = _matrix("A", A)
    N = _matrix("W", W)[0]
    code = _code("A", A.dtype)
    for name, t, shape in (("A", A, A.shape), ("W", W, (N, K)), ("dout", dout, (M, N))):
        _expect(name, t, shape, A.dtype, A.device)
    with _Launch(A, stream) as la:
        dA, dW = la.empty((M, K), A.dtype, needs[0]), la.empty((N, K), A.dtype, needs[1])
        dbias = la.empty((N,), torch.float32, bias)
        ws = la.workspace(lib.jepa_linear_bwd_workspace_bytes(M, N, K, code))
        check(lib.jepa_linear_bwd(_ptr(dout), _ptr(A), _ptr(W), _ptr(dA), _ptr(dW), _ptr(dbias), M, N, K, code,
                                  _ptr(ws), ws.numel(), la.handle))
    return dA, dW, dbias
