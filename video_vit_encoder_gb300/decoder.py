"""Python face of the decoder operators of the C ABI.

What training and serving a causal decoder on the encoder's tokens needs beside
``training.py``: the embedding of tokens and its gradient, the gated linear
recurrence forward, backward and one step at a time, and the distillation of a
linear classifier from a teacher's top logits.  Tensors, streams, workspaces and
errors are as there: contiguous tensors on one CUDA device, work enqueued on
``stream`` or on that device's current stream, outputs and workspaces allocated
on the stream that uses them, no part in autograd, and the first call of a
function on a device made outside a capture.
"""
from __future__ import annotations

import torch

from .training import (
    _CODE, _MOST, _a16, _c, _code, _elsewhere, _empty, _expect, _f32, _like, _matrix, _p, _place, _raw_stream, _u8,
    _workspace_bytes, check,
)

_i64, _i32 = torch.int64, torch.int32
SCAN_PIECE = 128   # JEPA_SCAN_PIECE of include/jepa_gb300.h: steps from one kept state to the next


def _ids(name, t, shape, device):
    """Token or class ids as int64."""
    if t.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"{name} are {t.dtype}: int64 or int32")
    _expect(name, t, shape, t.dtype, device)
    return t


# ----------------------------------------------------------------------------- embedding
def _embedding_types(table, out):
    tc, oc = _code("table", table), _code("out_dtype", out)
    if out != table and out != _f32:
        raise ValueError(f"rows of {out} with a table of {table}: equal, or rows in float32")
    return tc, oc


def _check_lookup(tokens, table, out_dtype):
    V, D = _matrix("table", table)
    _embedding_types(table.dtype, out_dtype)
    _expect("table", table, (V, D), table.dtype, table.device)
    _ids("tokens", tokens, tokens.shape, table.device)
    if tokens.numel() > _MOST:
        raise ValueError(f"tokens has shape {tuple(tokens.shape)}: at most {_MOST} tokens")


def embedding_fwd(tokens, table, scale=1.0, ignore_index=-100, out_dtype=None, stream=None):
    """scale * table[tokens], [..., dim]: tokens int64 (or int32) of any shape,
    table [vocab, dim]; out_dtype is the table's (default) or float32.  Tokens
    equal to ignore_index give zeros."""
    dt, dev, shape, n = table.dtype, table.device, table.shape, tokens.numel()
    out_dtype = out_dtype or dt
    tc, oc = _CODE.get(dt), _CODE.get(out_dtype)
    # one look at a usual call; anything else is told apart by _check_lookup
    if tc is None or (oc != tc and oc != 0) or tokens.dtype is not _i64 or n > _MOST or len(shape) != 2 or \
            max(shape) > _MOST or not table.is_contiguous() or not tokens.is_contiguous() or tokens.device != dev:
        _check_lookup(tokens, table, out_dtype)
    if _elsewhere(table, stream):
        with _place(table, stream, tokens):
            return embedding_fwd(tokens, table, scale, ignore_index, out_dtype)
    V, D = shape
    if tokens.dtype is not _i64:
        tokens = tokens.long()
    out = _empty(tokens.shape + (D,), dtype=out_dtype, device=dev)
    check(_c().jepa_embedding_fwd(tokens.data_ptr(), table.data_ptr(), out.data_ptr(), n, D, V, tc, oc, scale, ignore_index,
                                  _raw_stream(dev.index)))
    return out


def embedding_bwd(dout, tokens, vocab, scale=1.0, ignore_index=-100, out_dtype=None, stream=None):
    """The table's gradient [vocab, dim] from dout [..., dim] (the forward
    pass's output type); out_dtype is the table's type (default: dout's)."""
    dt, dev = dout.dtype, dout.device
    out_dtype = out_dtype or dt
    tc, oc = _embedding_types(out_dtype, dt)
    if dout.dim() < 1:
        raise ValueError("dout must have at least one dimension")
    D, n = dout.shape[-1], tokens.numel()
    if n > _MOST or D > _MOST or vocab > _MOST:
        raise ValueError(f"dout has shape {tuple(dout.shape)}, vocab {vocab}: at most {_MOST} tokens and columns, and rows")
    _expect("dout", dout, tokens.shape + (D,), dt, dev)
    _ids("tokens", tokens, tokens.shape, dev)
    if _elsewhere(dout, stream):
        with _place(dout, stream, tokens):
            return embedding_bwd(dout, tokens, vocab, scale, ignore_index, out_dtype)
    tok = tokens.long()
    dtable = _empty((vocab, D), dtype=out_dtype, device=dev)
    nb = _workspace_bytes("jepa_embedding_bwd_workspace_bytes", n, D, vocab)
    ws = _empty(nb, dtype=_u8, device=dev) if nb else None
    check(_c().jepa_embedding_bwd(tok.data_ptr(), dout.data_ptr(), dtable.data_ptr(), n, D, vocab, oc, tc, scale,
                                  ignore_index, _p(ws), nb, _raw_stream(dev.index)))
    return dtable


# ----------------------------------------------------------------------------- gated linear recurrence
def _scan_args(gv, lengths):
    shape, dt, dev = gv.shape, gv.dtype, gv.device
    if len(shape) != 3 or shape[2] % 2 or not shape[2]:
        raise ValueError(f"gv must be [batch, steps, 2 width], has shape {tuple(shape)}")
    B, T, C = shape[0], shape[1], shape[2] // 2
    if B > 65535 or B * T > _MOST or T > _MOST or C > 1 << 20:
        raise ValueError(f"gv has shape {tuple(shape)}: at most 65535 sequences, {_MOST} steps in all, width {1 << 20}")
    code = _code("gv", dt)
    if not gv.is_contiguous():
        raise ValueError("gv must be contiguous")
    if lengths is not None:
        _expect("lengths", lengths, (B,), _i32, dev)
    return B, T, C, dt, dev, code


def gated_scan_fwd(gv, h0=None, lengths=None, states=True, last=None, stream=None):
    """(h, last, states) of h_t = f_t h_{t-1} + (1 - f_t) v_t, f = sigmoid(g):
    gv [batch, steps, 2 width], gates then values; h0 float [batch, width] or
    None for zeros; lengths int32 [batch] or None.  h [batch, steps, width] in
    gv's dtype, zeros past a sequence's length; last float [batch, width], the
    states after the sequences (written into the argument if it is given; it may
    be h0); states float [batch, pieces, width], what gated_scan_bwd needs, or
    None if not asked for."""
    B, T, C, dt, dev, code = _scan_args(gv, lengths)
    if h0 is not None:
        _expect("h0", h0, (B, C), _f32, dev)
    if last is not None and last is not h0:
        _expect("last", last, (B, C), _f32, dev)
    if _elsewhere(gv, stream):
        with _place(gv, stream, h0, lengths, last):
            return gated_scan_fwd(gv, h0, lengths, states, last)
    h = _empty((B, T, C), dtype=dt, device=dev)
    if last is None:
        last = _empty((B, C), dtype=_f32, device=dev)
    kept = _empty((B, -(-T // SCAN_PIECE), C), dtype=_f32, device=dev) if states else None
    check(_c().jepa_gated_scan_fwd(gv.data_ptr(), _p(h0), _p(lengths), h.data_ptr(), last.data_ptr(), _p(kept), B, T, C,
                                   code, _raw_stream(dev.index)))
    return h, last, kept


def gated_scan_bwd(dh, gv, states, lengths=None, dlast=None, needs=True, stream=None):
    """(dgv, dh0) from dh [batch, steps, width] in gv's dtype, the forward
    pass's states, and dlast float [batch, width], the gradient of its last
    (None for zeros).  needs: whether dh0 is wanted."""
    B, T, C, dt, dev, code = _scan_args(gv, lengths)
    _expect("dh", dh, (B, T, C), dt, dev)
    _expect("states", states, (B, -(-T // SCAN_PIECE), C), _f32, dev)
    _expect("dlast", dlast, (B, C), _f32, dev)
    if _elsewhere(gv, stream):
        with _place(gv, stream, dh, states, lengths, dlast):
            return gated_scan_bwd(dh, gv, states, lengths, dlast, needs)
    dgv = _like(gv)
    dh0 = _empty((B, C), dtype=_f32, device=dev) if needs else None
    check(_c().jepa_gated_scan_bwd(dh.data_ptr(), gv.data_ptr(), states.data_ptr(), _p(lengths), _p(dlast),
                                   dgv.data_ptr(), _p(dh0), B, T, C, code, _raw_stream(dev.index)))
    return dgv, dh0


# ----------------------------------------------------------------------------- distillation
def _distill_args(x, W, bias, top_logits, top_ids):
    M, D = _matrix("x", x)
    V = _matrix("W", W)[0]
    K = _matrix("top_ids", top_ids)[1]
    dt, dev = x.dtype, x.device
    code, tcode = _code("x", dt), _code("top_logits", top_logits.dtype)
    _expect("x", x, (M, D), dt, dev)
    _expect("W", W, (V, D), dt, dev)
    _expect("bias", bias, (V,), _f32, dev)
    _ids("top_ids", top_ids, (M, K), dev)
    _expect("top_logits", top_logits, (M, K), top_logits.dtype, dev)
    return M, D, V, K, code, tcode


def linear_distill_fwd(x, W, bias, top_logits, top_ids, temperature=1.0, ignore_index=-100, stream=None):
    """(loss, lse, z): the loss float [M] of the classifier x W^T + bias against
    a teacher of whom the K best logits are known, tau^2 KL(softmax(top_logits /
    tau) | softmax(z / tau)); lse float [M] and z float [M, K], the student's
    logits of the entries, are for the backward pass.  x [M, D], W [V, D] in one
    dtype, bias float [V] or None; top_logits [M, K] of any of the dtypes,
    top_ids int64 (or int32) [M, K].  Entries with id ignore_index are out; a
    row without entries has loss 0."""
    M, D, V, K, code, tcode = _distill_args(x, W, bias, top_logits, top_ids)
    if _elsewhere(x, stream):
        with _place(x, stream, W, bias, top_logits, top_ids):
            return linear_distill_fwd(x, W, bias, top_logits, top_ids, temperature, ignore_index)
    dev = x.device
    ids, x, W = top_ids.long(), _a16(x), _a16(W)
    loss = _empty(M, dtype=_f32, device=dev)
    lse = _like(loss)
    z = _empty((M, K), dtype=_f32, device=dev)
    n = _workspace_bytes("jepa_linear_distill_workspace_bytes", M, D, V, K, code, 0)
    ws = _empty(n, dtype=_u8, device=dev)
    check(_c().jepa_linear_distill_fwd(x.data_ptr(), W.data_ptr(), _p(bias), top_logits.data_ptr(), ids.data_ptr(),
                                       loss.data_ptr(), lse.data_ptr(), z.data_ptr(), M, D, V, K, code, tcode,
                                       ignore_index, temperature, ws.data_ptr(), n, _raw_stream(dev.index)))
    return loss, lse, z


def linear_distill_bwd(dloss, x, W, bias, top_logits, top_ids, lse, z, temperature=1.0, ignore_index=-100,
                       needs=(True, True, True), stream=None):
    """(dx, dW, dbias) from dloss, the gradient of each row's loss (float [M],
    or one number for all rows: 1 / n for the mean of n rows), and the forward
    pass's lse and z.  needs: (dx, dW, dbias).  In 16 bits the logits' gradient
    is rounded to the type between the products, so that dx and dW carry one
    rounding more than their own; in float32 it is not."""
    M, D, V, K, code, tcode = _distill_args(x, W, bias, top_logits, top_ids)
    dev = x.device
    _expect("lse", lse, (M,), _f32, dev)
    _expect("z", z, (M, K), _f32, dev)
    if _elsewhere(x, stream):
        with _place(x, stream, dloss, W, bias, top_logits, top_ids, lse, z):
            return linear_distill_bwd(dloss, x, W, bias, top_logits, top_ids, lse, z, temperature, ignore_index, needs)
    if not torch.is_tensor(dloss):
        dloss = torch.full((M,), float(dloss), device=dev)
    elif dloss.dim() == 0:
        dloss = dloss.to(device=dev, dtype=_f32).expand(M).contiguous()
    _expect("dloss", dloss, (M,), _f32, dev)
    ids, x, W = top_ids.long(), _a16(x), _a16(W)
    dx = _like(x) if needs[0] else None
    dW = _like(W) if needs[1] else None
    db = _empty(V, dtype=_f32, device=dev) if needs[2] else None
    n = _workspace_bytes("jepa_linear_distill_workspace_bytes", M, D, V, K, code, 1)
    ws = _empty(n, dtype=_u8, device=dev)
    check(_c().jepa_linear_distill_bwd(x.data_ptr(), W.data_ptr(), _p(bias), top_logits.data_ptr(), ids.data_ptr(),
                                       lse.data_ptr(), z.data_ptr(), dloss.data_ptr(), _p(dx), _p(dW), _p(db), M, D, V, K,
                                       code, tcode, ignore_index, temperature, ws.data_ptr(), n,
                                       _raw_stream(dev.index)))
    return dx, dW, db
