"""Python face of the training operators of the C ABI.

Layer norm, gated feed-forward, softmax cross entropy of a linear classifier
and the linear layer, each as a forward and a backward function (the linear
layer's forward pass is ``linear``).  Every computation runs in
libjepa_gb300.so; torch supplies device memory and streams.  The functions take
no part in autograd: results carry no graph, whatever the arguments require.

Tensors are contiguous and on one CUDA device, which need not be the current
one; row counts and widths are at most 2^24 (layer norm's width: 2^20).  Work is
enqueued on ``stream``, or on that device's current stream; the outputs and the
workspace are allocated on the stream that uses them, so calls on several
streams, and captured graphs, never share one.  ``stream`` has to have waited for
whatever wrote the inputs; they may be dropped as soon as the call returns.
Gradients not asked for (``needs``) are returned as None.  The first call of a
function on a device is made outside a capture.
"""
from __future__ import annotations

import contextlib
import functools

import torch

from . import _lib
from ._lib import check, load
from .binding import DTYPE_CODE

_CODE = {torch.float32: DTYPE_CODE["f32"], torch.float16: DTYPE_CODE["f16"], torch.bfloat16: DTYPE_CODE["bf16"]}
# the handle of a device's current stream, and the current device (calls a fifth as long as through torch.cuda)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_empty, _like = torch.empty, torch.empty_like   # _like takes half the time
_f32, _u8 = torch.float32, torch.uint8
_ACT = {"silu": _lib.GATE_SILU, "gelu": _lib.GATE_GELU}


def _expect(name, t, shape, dtype, device):
    """t is None or a contiguous tensor of this shape, dtype and device."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


# the library's limit on row counts and widths; it takes them as C ints, into which a larger one may not be squeezed
_MOST = 1 << 24


def _matrix(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, has shape {tuple(t.shape)}")
    if max(t.shape) > _MOST:
        raise ValueError(f"{name} has shape {tuple(t.shape)}: at most {_MOST} rows and columns")
    return t.shape


def _rows(shape):
    """The leading shape, its number of rows and the last dimension of x's."""
    if not shape:
        raise ValueError("x must have at least one dimension")
    lead = shape[:-1]
    rows, dim = lead.numel(), shape[-1]
    if rows > _MOST or dim > _MOST:
        raise ValueError(f"x has shape {tuple(shape)}: at most {_MOST} rows and columns")
    return lead, rows, dim


def _code(name, dtype):
    code = _CODE.get(dtype)
    if code is None:
        raise ValueError(f"{name} is {dtype}: float32, float16 or bfloat16")
    return code


def _c():
    """The library, loaded on the first call."""
    return _lib._lib or load()


def _p(t):
    return None if t is None else t.data_ptr()


def _a16(t):
    """The matrix, or a copy of one that does not start on 16 bytes (a view
    into another tensor can start anywhere)."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(query, *sizes):
    return getattr(load(), query)(*sizes)


@contextlib.contextmanager
def _place(t, stream, *inputs):
    """t's device and the stream current, so that what a call allocates
    belongs to the stream that uses it; the memory of t and of the other inputs
    is not given out again before the stream is done with it."""
    if t.get_device() < 0:
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
    if stream is not None and stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, tensors are on {t.device}")
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        yield
    if stream is not None:
        for i in (t,) + inputs:
            if torch.is_tensor(i) and i.is_cuda:
                i.record_stream(stream)


def _elsewhere(t, stream):
    """Whether a call on t has to be made under _place (which refuses CPU tensors)."""
    index = t.get_device()
    return stream is not None or index < 0 or index != _current_device()


def layernorm_fwd(x, w, b, eps, out_dtype=None, stream=None):
    """(y, mean, rstd) of x [..., dim] over its last dimension; w, b float
    [dim].  y has out_dtype (default x's; another one needs float32 x), mean
    and rstd are float32 of x's leading shape."""
    shape, dt, dev = x.shape, x.dtype, x.device
    lead, rows, dim = _rows(shape)
    out_dtype = out_dtype or dt
    xc, yc = _code("x", dt), _code("out_dtype", out_dtype)
    _expect("x", x, shape, dt, dev)
    _expect("w", w, (dim,), _f32, dev)
    _expect("b", b, (dim,), _f32, dev)
    if _elsewhere(x, stream):
        with _place(x, stream, w, b):
            return layernorm_fwd(x, w, b, eps, out_dtype)
    y = _like(x, dtype=out_dtype)
    mean = _empty(lead, dtype=_f32, device=dev)
    rstd = _like(mean)
    check(_c().jepa_layernorm_fwd(x.data_ptr(), w.data_ptr(), b.data_ptr(), y.data_ptr(), mean.data_ptr(),
                                  rstd.data_ptr(), rows, dim, xc, yc, eps, _raw_stream(dev.index)))
    return y, mean, rstd


def layernorm_bwd(dy, x, w, mean, rstd, residual=None, needs=(True, True), stream=None):
    """(dx, dw, db) from dy (y's shape and dtype), x, w and the forward pass's
    mean and rstd.  residual: x's shape and dtype, added to dx.  needs: (dw,
    db)."""
    shape, dt, dev = x.shape, x.dtype, x.device
    lead, rows, dim = _rows(shape)
    xc, yc = _code("x", dt), _code("dy", dy.dtype)
    _expect("x", x, shape, dt, dev)
    _expect("dy", dy, shape, dy.dtype, dev)
    _expect("w", w, (dim,), _f32, dev)
    _expect("mean", mean, lead, _f32, dev)
    _expect("rstd", rstd, lead, _f32, dev)
    _expect("residual", residual, shape, dt, dev)
    if _elsewhere(x, stream):
        with _place(x, stream, dy, w, mean, rstd, residual):
            return layernorm_bwd(dy, x, w, mean, rstd, residual, needs)
    dx = _like(x)
    dw = _like(w) if needs[0] else None
    db = _like(w) if needs[1] else None
    n = _workspace_bytes("jepa_layernorm_bwd_workspace_bytes", rows, dim)
    ws = _empty(n, dtype=_u8, device=dev)
    check(_c().jepa_layernorm_bwd(dy.data_ptr(), x.data_ptr(), w.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                  _p(residual), dx.data_ptr(), _p(dw), _p(db), rows, dim, xc, yc, ws.data_ptr(), n,
                                  _raw_stream(dev.index)))
    return dx, dw, db


def _ce_args(x, W, bias, labels):
    M, D = _matrix("x", x)
    V = _matrix("W", W)[0]
    dt, dev = x.dtype, x.device
    code = _code("x", dt)
    _expect("x", x, (M, D), dt, dev)
    _expect("W", W, (V, D), dt, dev)
    _expect("bias", bias, (V,), _f32, dev)
    if labels.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"labels are {labels.dtype}: int64 or int32")
    _expect("labels", labels, (M,), labels.dtype, dev)
    return M, D, V, code


def linear_ce_fwd(x, W, bias, labels, ignore_index=-100, smoothing=0.0, stream=None):
    """(loss, lse), float [M], of the classifier x W^T + bias: x [M, D], W
    [V, D] in one dtype, bias float [V] or None, labels int64 (or int32) [M].
    Rows with label ignore_index have loss 0."""
    M, D, V, code = _ce_args(x, W, bias, labels)
    if _elsewhere(x, stream):
        with _place(x, stream, W, bias, labels):
            return linear_ce_fwd(x, W, bias, labels, ignore_index, smoothing)
    dev = x.device
    lab, x, W = labels.long(), _a16(x), _a16(W)
    loss = _empty(M, dtype=_f32, device=dev)
    lse = _like(loss)
    n = _workspace_bytes("jepa_linear_ce_workspace_bytes", M, D, V, code, 0)
    ws = _empty(n, dtype=_u8, device=dev)
    check(_c().jepa_linear_ce_fwd(x.data_ptr(), W.data_ptr(), _p(bias), lab.data_ptr(), loss.data_ptr(),
                                  lse.data_ptr(), M, D, V, code, ignore_index, smoothing, ws.data_ptr(), n,
                                  _raw_stream(dev.index)))
    return loss, lse


def linear_ce_bwd(dloss, x, W, bias, labels, lse, ignore_index=-100, smoothing=0.0, needs=(True, True, True),
                  stream=None):
    """(dx, dW, dbias) from dloss, the gradient of each row's loss (float [M],
    or one number for all rows: 1 / n for the mean of n rows), and the forward
    pass's lse.  needs: (dx, dW, dbias)."""
    M, D, V, code = _ce_args(x, W, bias, labels)
    _expect("lse", lse, (M,), _f32, x.device)
    if _elsewhere(x, stream):
        with _place(x, stream, dloss, W, bias, labels, lse):
            return linear_ce_bwd(dloss, x, W, bias, labels, lse, ignore_index, smoothing, needs)
    dev = x.device
    if not torch.is_tensor(dloss):
        dloss = torch.full((M,), float(dloss), device=dev)
    elif dloss.dim() == 0:
        dloss = dloss.to(device=dev, dtype=_f32).expand(M).contiguous()
    _expect("dloss", dloss, (M,), _f32, dev)
    lab, x, W = labels.long(), _a16(x), _a16(W)
    dx = _like(x) if needs[0] else None
    dW = _like(W) if needs[1] else None
    db = _empty(V, dtype=_f32, device=dev) if needs[2] else None
    n = _workspace_bytes("jepa_linear_ce_workspace_bytes", M, D, V, code, 1)
    ws = _empty(n, dtype=_u8, device=dev)
    check(_c().jepa_linear_ce_bwd(x.data_ptr(), W.data_ptr(), _p(bias), lab.data_ptr(), lse.data_ptr(),
                                  dloss.data_ptr(), _p(dx), _p(dW), _p(db), M, D, V, code, ignore_index, smoothing,
                                  ws.data_ptr(), n, _raw_stream(dev.index)))
    return dx, dW, db


def _ffn_args(x, Wg, Wu, bg, bu, act):
    M, D = _matrix("x", x)
    F = _matrix("Wg", Wg)[0]
    dt, dev = x.dtype, x.device
    code = _code("x", dt)
    _expect("x", x, (M, D), dt, dev)
    _expect("Wg", Wg, (F, D), dt, dev)
    _expect("Wu", Wu, (F, D), dt, dev)
    _expect("bg", bg, (F,), _f32, dev)
    _expect("bu", bu, (F,), _f32, dev)
    if act not in _ACT:
        raise ValueError(f"act {act!r}: 'silu' or 'gelu'")
    return M, D, F, code, _ACT[act]


def gated_ffn_fwd(x, Wg, Wu, bg=None, bu=None, act="silu", stream=None):
    """h = act(x Wg^T + bg) * (x Wu^T + bu), [M, F] in x's dtype: x [M, D],
    Wg, Wu [F, D]; bg, bu float [F] or None; act 'silu' or 'gelu' (erf)."""
    M, D, F, code, a = _ffn_args(x, Wg, Wu, bg, bu, act)
    if _elsewhere(x, stream):
        with _place(x, stream, Wg, Wu, bg, bu):
            return gated_ffn_fwd(x, Wg, Wu, bg, bu, act)
    dev = x.device
    x, Wg, Wu = _a16(x), _a16(Wg), _a16(Wu)
    h = _empty((M, F), dtype=x.dtype, device=dev)
    n = _workspace_bytes("jepa_gated_ffn_workspace_bytes", M, D, F, code, 0)
    ws = _empty(n, dtype=_u8, device=dev) if n else None
    check(_c().jepa_gated_ffn_fwd(x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), _p(bg), _p(bu), h.data_ptr(), M, D, F,
                                  code, a, _p(ws), n, _raw_stream(dev.index)))
    return h


def gated_ffn_bwd(dh, x, Wg, Wu, bg=None, bu=None, act="silu", needs=(True, True, True, True, True), stream=None):
    """(dx, dWg, dWu, dbg, dbu) from dh [M, F]; the projections are computed
    again from x.  needs: one flag for each."""
    M, D, F, code, a = _ffn_args(x, Wg, Wu, bg, bu, act)
    _expect("dh", dh, (M, F), x.dtype, x.device)
    if _elsewhere(x, stream):
        with _place(x, stream, dh, Wg, Wu, bg, bu):
            return gated_ffn_bwd(dh, x, Wg, Wu, bg, bu, act, needs)
    dev = x.device
    dh, x, Wg, Wu = _a16(dh), _a16(x), _a16(Wg), _a16(Wu)
    dx = _like(x) if needs[0] else None
    dWg = _like(Wg) if needs[1] else None
    dWu = _like(Wu) if needs[2] else None
    dbg = _empty(F, dtype=_f32, device=dev) if needs[3] else None
    dbu = _empty(F, dtype=_f32, device=dev) if needs[4] else None
    n = _workspace_bytes("jepa_gated_ffn_workspace_bytes", M, D, F, code, 1)
    ws = _empty(n, dtype=_u8, device=dev)
    check(_c().jepa_gated_ffn_bwd(dh.data_ptr(), x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), _p(bg), _p(bu), _p(dx),
                                  _p(dWg), _p(dWu), _p(dbg), _p(dbu), M, D, F, code, a, ws.data_ptr(), n,
                                  _raw_stream(dev.index)))
    return dx, dWg, dWu, dbg, dbu


def linear_bwd(dout, A, W, bias=True, needs=(True, True), stream=None):
    """(dA, dW, dbias) of out = A W^T + bias from dout [M, N]: A [M, K], W
    [N, K] and dout in one dtype.  needs: (dA, dW); bias: whether dbias (float
    [N]) is wanted."""
    M, K = _matrix("A", A)
    N = _matrix("W", W)[0]
    dt, dev = A.dtype, A.device
    code = _code("A", dt)
    _expect("A", A, (M, K), dt, dev)
    _expect("W", W, (N, K), dt, dev)
    _expect("dout", dout, (M, N), dt, dev)
    if _elsewhere(A, stream):
        with _place(A, stream, dout, W):
            return linear_bwd(dout, A, W, bias, needs)
    dout, A, W = _a16(dout), _a16(A), _a16(W)
    dA = _like(A) if needs[0] else None
    dW = _like(W) if needs[1] else None
    db = _empty(N, dtype=_f32, device=dev) if bias else None
    n = _workspace_bytes("jepa_linear_bwd_workspace_bytes", M, N, K, code)
    ws = _empty(n, dtype=_u8, device=dev) if n else None
    check(_c().jepa_linear_bwd(dout.data_ptr(), A.data_ptr(), W.data_ptr(), _p(dA), _p(dW), _p(db), M, N, K, code,
                               _p(ws), n, _raw_stream(dev.index)))
    return dA, dW, db
