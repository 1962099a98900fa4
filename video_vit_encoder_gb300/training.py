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

import functools

import torch

from . import _lib
from ._lib import check, load
from .binding import DTYPE_CODE

_CODE = {torch.float32: DTYPE_CODE["f32"], torch.float16: DTYPE_CODE["f16"], torch.bfloat16: DTYPE_CODE["bf16"]}
# the handle of a device's current stream (a call a fifth as long as through torch.cuda.current_stream)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_empty = torch.empty
_f32 = torch.float32
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


def _matrix(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, has shape {tuple(t.shape)}")
    return t.shape


def _code(name, dtype):
    code = _CODE.get(dtype)
    if code is None:
        raise ValueError(f"{name} is {dtype}: float32, float16 or bfloat16")
    return code


def _p(t):
    return None if t is None else t.data_ptr()


def _a16(t):
    """The matrix, or a copy of one that does not start on 16 bytes (a view
    into another tensor can start anywhere)."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(query, *sizes):
    return getattr(load(), query)(*sizes)


def _run(t, stream, body):
    """body(device, stream handle) with t's device and the stream current, so
    that what it allocates belongs to the stream that uses it."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
    if stream is None:
        if index == torch.cuda.current_device():
            return body(t.device, _raw_stream(index))
        with torch.cuda.device(index):
            return body(t.device, _raw_stream(index))
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, tensors are on {t.device}")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return body(t.device, stream.cuda_stream)


def layernorm_fwd(x, w, b, eps, out_dtype=None, stream=None):
    """(y, mean, rstd) of x [..., dim] over its last dimension; w, b float
    [dim].  y has out_dtype (default x's; another one needs float32 x), mean
    and rstd are float32 of x's leading shape."""
    lib = load()
    shape, dt = x.shape, x.dtype
    dim = shape[-1]
    out_dtype = out_dtype or dt
    xc, yc = _code("x", dt), _code("out_dtype", out_dtype)
    dev = x.device
    _expect("x", x, shape, dt, dev)
    _expect("w", w, (dim,), _f32, dev)
    _expect("b", b, (dim,), _f32, dev)

    def body(dev, handle):
        lead = shape[:-1]
        rows = lead.numel()
        y = _empty(shape, dtype=out_dtype, device=dev)
        mean, rstd = _empty(lead, dtype=_f32, device=dev), _empty(lead, dtype=_f32, device=dev)
        check(lib.jepa_layernorm_fwd(_p(x), _p(w), _p(b), _p(y), _p(mean), _p(rstd), rows, dim, xc, yc, eps, handle))
        return y, mean, rstd
    return _run(x, stream, body)


def layernorm_bwd(dy, x, w, mean, rstd, residual=None, needs=(True, True), stream=None):
    """(dx, dw, db) from dy (y's shape and dtype), x, w and the forward pass's
    mean and rstd.  residual: x's shape and dtype, added to dx.  needs: (dw,
    db)."""
    lib = load()
    shape, dt, dev = x.shape, x.dtype, x.device
    dim, lead = shape[-1], shape[:-1]
    xc, yc = _code("x", dt), _code("dy", dy.dtype)
    _expect("x", x, shape, dt, dev)
    _expect("dy", dy, shape, dy.dtype, dev)
    _expect("w", w, (dim,), _f32, dev)
    _expect("mean", mean, lead, _f32, dev)
    _expect("rstd", rstd, lead, _f32, dev)
    _expect("residual", residual, shape, dt, dev)

    def body(dev, handle):
        rows = lead.numel()
        dx = _empty(shape, dtype=dt, device=dev)
        dw = _empty(dim, dtype=_f32, device=dev) if needs[0] else None
        db = _empty(dim, dtype=_f32, device=dev) if needs[1] else None
        n = _workspace_bytes("jepa_layernorm_bwd_workspace_bytes", rows, dim)
        ws = _empty(n, dtype=torch.uint8, device=dev)
        check(lib.jepa_layernorm_bwd(_p(dy), _p(x), _p(w), _p(mean), _p(rstd), _p(residual), _p(dx), _p(dw), _p(db),
                                     rows, dim, xc, yc, _p(ws), n, handle))
        return dx, dw, db
    return _run(x, stream, body)


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
    lib = load()
    M, D, V, code = _ce_args(x, W, bias, labels)

    def body(dev, handle):
        lab, xx, ww = labels.long(), _a16(x), _a16(W)
        loss, lse = _empty(M, dtype=_f32, device=dev), _empty(M, dtype=_f32, device=dev)
        n = _workspace_bytes("jepa_linear_ce_workspace_bytes", M, D, V, code, 0)
        ws = _empty(n, dtype=torch.uint8, device=dev)
        check(lib.jepa_linear_ce_fwd(_p(xx), _p(ww), _p(bias), _p(lab), _p(loss), _p(lse), M, D, V, code, ignore_index,
                                     smoothing, _p(ws), n, handle))
        return loss, lse
    return _run(x, stream, body)


def linear_ce_bwd(dloss, x, W, bias, labels, lse, ignore_index=-100, smoothing=0.0, needs=(True, True, True),
                  stream=None):
    """(dx, dW, dbias) from dloss, the gradient of each row's loss (float [M],
    or one number for all rows: 1 / n for the mean of n rows), and the forward
    pass's lse.  needs: (dx, dW, dbias)."""
    lib = load()
    M, D, V, code = _ce_args(x, W, bias, labels)
    _expect("lse", lse, (M,), _f32, x.device)

    def body(dev, handle):
        lab, dl, dt, xx, ww = labels.long(), dloss, x.dtype, _a16(x), _a16(W)
        if not torch.is_tensor(dl):
            dl = torch.full((M,), float(dl), device=dev)
        elif dl.dim() == 0:
            dl = dl.to(device=dev, dtype=_f32).expand(M).contiguous()
        _expect("dloss", dl, (M,), _f32, dev)
        dx = _empty((M, D), dtype=dt, device=dev) if needs[0] else None
        dW = _empty((V, D), dtype=dt, device=dev) if needs[1] else None
        db = _empty(V, dtype=_f32, device=dev) if needs[2] else None
        n = _workspace_bytes("jepa_linear_ce_workspace_bytes", M, D, V, code, 1)
        ws = _empty(n, dtype=torch.uint8, device=dev)
        check(lib.jepa_linear_ce_bwd(_p(xx), _p(ww), _p(bias), _p(lab), _p(lse), _p(dl), _p(dx), _p(dW), _p(db), M, D, V,
                                     code, ignore_index, smoothing, _p(ws), n, handle))
        return dx, dW, db
    return _run(x, stream, body)


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
    lib = load()
    M, D, F, code, a = _ffn_args(x, Wg, Wu, bg, bu, act)

    def body(dev, handle):
        xx, wg, wu = _a16(x), _a16(Wg), _a16(Wu)
        h = _empty((M, F), dtype=x.dtype, device=dev)
        n = _workspace_bytes("jepa_gated_ffn_workspace_bytes", M, D, F, code, 0)
        ws = _empty(n, dtype=torch.uint8, device=dev) if n else None
        check(lib.jepa_gated_ffn_fwd(_p(xx), _p(wg), _p(wu), _p(bg), _p(bu), _p(h), M, D, F, code, a, _p(ws), n, handle))
        return h
    return _run(x, stream, body)


def gated_ffn_bwd(dh, x, Wg, Wu, bg=None, bu=None, act="silu", needs=(True, True, True, True, True), stream=None):
    """(dx, dWg, dWu, dbg, dbu) from dh [M, F]; the projections are computed
    again from x.  needs: one flag for each."""
    lib = load()
    M, D, F, code, a = _ffn_args(x, Wg, Wu, bg, bu, act)
    _expect("dh", dh, (M, F), x.dtype, x.device)

    def body(dev, handle):
        dt, d, xx, wg, wu = x.dtype, _a16(dh), _a16(x), _a16(Wg), _a16(Wu)
        dx = _empty((M, D), dtype=dt, device=dev) if needs[0] else None
        dWg = _empty((F, D), dtype=dt, device=dev) if needs[1] else None
        dWu = _empty((F, D), dtype=dt, device=dev) if needs[2] else None
        dbg = _empty(F, dtype=_f32, device=dev) if needs[3] else None
        dbu = _empty(F, dtype=_f32, device=dev) if needs[4] else None
        n = _workspace_bytes("jepa_gated_ffn_workspace_bytes", M, D, F, code, 1)
        ws = _empty(n, dtype=torch.uint8, device=dev)
        check(lib.jepa_gated_ffn_bwd(_p(d), _p(xx), _p(wg), _p(wu), _p(bg), _p(bu), _p(dx), _p(dWg), _p(dWu), _p(dbg),
                                     _p(dbu), M, D, F, code, a, _p(ws), n, handle))
        return dx, dWg, dWu, dbg, dbu
    return _run(x, stream, body)


def linear_bwd(dout, A, W, bias=True, needs=(True, True), stream=None):
    """(dA, dW, dbias) of out = A W^T + bias from dout [M, N]: A [M, K], W
    [N, K] and dout in one dtype.  needs: (dA, dW); bias: whether dbias (float
    [N]) is wanted."""
    lib = load()
    M, K = _matrix("A", A)
    N = _matrix("W", W)[0]
    dt, dev = A.dtype, A.device
    code = _code("A", dt)
    _expect("A", A, (M, K), dt, dev)
    _expect("W", W, (N, K), dt, dev)
    _expect("dout", dout, (M, N), dt, dev)

    def body(dev, handle):
        d, a, w = _a16(dout), _a16(A), _a16(W)
        dA = _empty((M, K), dtype=dt, device=dev) if needs[0] else None
        dW = _empty((N, K), dtype=dt, device=dev) if needs[1] else None
        db = _empty(N, dtype=_f32, device=dev) if bias else None
        n = _workspace_bytes("jepa_linear_bwd_workspace_bytes", M, N, K, code)
        ws = _empty(n, dtype=torch.uint8, device=dev) if n else None
        check(lib.jepa_linear_bwd(_p(d), _p(a), _p(w), _p(dA), _p(dW), _p(db), M, N, K, code, _p(ws), n, handle))
        return dA, dW, db
    return _run(A, stream, body)
