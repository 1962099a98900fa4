"""Refusals of the training operators, on the host: nothing here needs a GPU
(arguments are checked before anything is enqueued)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from video_vit_encoder_gb300 import build
    build.build()
    import video_vit_encoder_gb300 as jg
    return jg.load()


V = C.c_void_p(1 << 20)
ODD = C.c_void_p((1 << 20) + 1)
WS = C.c_void_p(1 << 20)
BIG = 1 << 40


def test_layernorm_refusals(lib):
    from video_vit_encoder_gb300._lib import ERR_ARG, ERR_UNSUPPORTED, OK

    def fwd(x=V, w=V, b=V, y=V, rows=4, dim=100, xt=0, yt=0, eps=1e-6):
        return lib.jepa_layernorm_fwd(x, w, b, y, V, V, rows, dim, xt, yt, eps, None)
    assert fwd(x=None, rows=0) == OK
    assert fwd(x=None) == fwd(w=None) == fwd(b=None) == fwd(y=None) == ERR_ARG
    assert fwd(rows=-1) == fwd(dim=0) == fwd(dim=(1 << 20) + 1) == fwd(rows=(1 << 24) + 1) == ERR_ARG
    assert fwd(xt=3) == fwd(yt=-1) == fwd(eps=0.0) == fwd(eps=float("nan")) == ERR_ARG
    assert fwd(xt=2, yt=0) == fwd(xt=1, yt=2) == ERR_UNSUPPORTED
    assert fwd(x=ODD) == fwd(w=ODD) == fwd(y=ODD) == ERR_ARG
    assert b"aligned" in lib.jepa_last_error()

    def bwd(dy=V, x=V, w=V, mean=V, rstd=V, res=None, dx=V, rows=4, dim=100, xt=0, yt=0, ws=WS, n=BIG):
        return lib.jepa_layernorm_bwd(dy, x, w, mean, rstd, res, dx, V, V, rows, dim, xt, yt, ws, n, None)
    for k in ("dy", "x", "w", "mean", "rstd", "dx"):
        assert bwd(**{k: None}) == ERR_ARG, k
        assert bwd(**{k: ODD}) == ERR_ARG, k
    assert bwd(res=ODD) == bwd(ws=None) == bwd(ws=C.c_void_p((1 << 20) + 16)) == ERR_ARG
    need = lib.jepa_layernorm_bwd_workspace_bytes(4, 100)
    assert need > 0 and bwd(n=need - 1) == ERR_ARG and b"workspace" in lib.jepa_last_error()
    assert lib.jepa_layernorm_bwd_workspace_bytes(-1, 100) == 0
    assert lib.jepa_layernorm_bwd_workspace_bytes(0, 100) == 0


def test_cross_entropy_refusals(lib):
    from video_vit_encoder_gb300._lib import ERR_ARG, OK

    def fwd(x=V, W=V, bias=None, lab=V, loss=V, lse=V, M=4, D=64, n=10, dt=2, s=0.0, ws=WS, nb=BIG):
        return lib.jepa_linear_ce_fwd(x, W, bias, lab, loss, lse, M, D, n, dt, -100, s, ws, nb, None)
    assert fwd(x=None, M=0) == OK
    for k in ("x", "W", "lab", "lse"):
        assert fwd(**{k: None}) == ERR_ARG, k
    for k in ("x", "W", "lab", "lse", "loss", "bias"):
        assert fwd(**{k: ODD}) == ERR_ARG, k
    assert fwd(lab=C.c_void_p((1 << 20) + 4)) == ERR_ARG
    assert fwd(M=-1) == fwd(D=0) == fwd(n=0) == fwd(n=(1 << 24) + 1) == fwd(dt=3) == ERR_ARG
    assert fwd(s=-0.1) == fwd(s=1.0) == fwd(s=float("nan")) == ERR_ARG
    need = lib.jepa_linear_ce_workspace_bytes(4, 64, 10, 2, 0)
    assert need > 0 and fwd(nb=need - 1) == fwd(ws=None) == ERR_ARG

    def bwd(x=V, W=V, bias=None, lab=V, lse=V, dl=V, dx=V, dW=V, db=V, M=4, D=64, n=10, dt=2, s=0.0, ws=WS, nb=BIG):
        return lib.jepa_linear_ce_bwd(x, W, bias, lab, lse, dl, dx, dW, db, M, D, n, dt, -100, s, ws, nb, None)
    for k in ("x", "W", "lab", "lse", "dl"):
        assert bwd(**{k: None}) == ERR_ARG, k
    for k in ("x", "W", "lab", "lse", "dl", "dx", "dW", "db", "bias"):
        assert bwd(**{k: ODD}) == ERR_ARG, k
    assert bwd(dx=None, dW=None, db=None) == ERR_ARG
    assert b"gradient" in lib.jepa_last_error()
    need = lib.jepa_linear_ce_workspace_bytes(4, 64, 10, 2, 1)
    assert need > 0 and bwd(nb=need - 1) == bwd(ws=None) == bwd(s=2.0) == ERR_ARG
    assert lib.jepa_linear_ce_workspace_bytes(4, 0, 10, 2, 1) == 0


def test_gated_ffn_refusals(lib):
    from video_vit_encoder_gb300._lib import ERR_ARG, OK

    def fwd(x=V, Wg=V, Wu=V, bg=None, bu=None, h=V, M=4, D=64, F=32, dt=2, act=0, ws=WS, nb=BIG):
        return lib.jepa_gated_ffn_fwd(x, Wg, Wu, bg, bu, h, M, D, F, dt, act, ws, nb, None)
    assert fwd(x=None, M=0) == OK
    for k in ("x", "Wg", "Wu", "h"):
        assert fwd(**{k: None}) == ERR_ARG, k
    for k in ("x", "Wg", "Wu", "h", "bg", "bu"):
        assert fwd(**{k: ODD}) == ERR_ARG, k
    assert fwd(M=-1) == fwd(D=0) == fwd(F=0) == fwd(dt=-1) == fwd(act=2) == fwd(act=-1) == ERR_ARG

    def bwd(dh=V, x=V, Wg=V, Wu=V, bg=None, bu=None, dx=V, dWg=V, dWu=V, dbg=V, dbu=V, M=4, D=64, F=32, dt=2, act=0,
            ws=WS, nb=BIG):
        return lib.jepa_gated_ffn_bwd(dh, x, Wg, Wu, bg, bu, dx, dWg, dWu, dbg, dbu, M, D, F, dt, act, ws, nb, None)
    for k in ("dh", "x", "Wg", "Wu"):
        assert bwd(**{k: None}) == ERR_ARG, k
    for k in ("dh", "x", "Wg", "Wu", "bg", "bu", "dx", "dWg", "dWu", "dbg", "dbu"):
        assert bwd(**{k: ODD}) == ERR_ARG, k
    assert bwd(dx=None, dWg=None, dWu=None, dbg=None, dbu=None) == bwd(act=7) == ERR_ARG
    need = lib.jepa_gated_ffn_workspace_bytes(4, 64, 32, 2, 1)
    assert need > 0 and bwd(nb=need - 1) == bwd(ws=None) == ERR_ARG


def test_linear_bwd_refusals(lib):
    from video_vit_encoder_gb300._lib import ERR_ARG

    def bwd(d=V, A=V, W=V, dA=V, dW=V, db=V, M=4, N=64, K=32, dt=2, ws=WS, nb=BIG):
        return lib.jepa_linear_bwd(d, A, W, dA, dW, db, M, N, K, dt, ws, nb, None)
    assert bwd(d=None) == bwd(A=None) == bwd(W=None) == bwd(dA=None, dW=None, db=None) == ERR_ARG
    for k in ("d", "A", "W", "dA", "dW", "db"):
        assert bwd(**{k: ODD}) == ERR_ARG, k
    assert bwd(M=-1) == bwd(N=0) == bwd(K=0) == bwd(dt=5) == bwd(K=(1 << 24) + 1) == ERR_ARG


def test_binding_refusals():
    """Shapes, dtypes, layout and device are refused before the library is called."""
    import video_vit_encoder_gb300 as jg
    x, W = torch.zeros(4, 8), torch.zeros(6, 8)
    lab = torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    bad = [
        lambda: jg.layernorm_fwd(x, torch.zeros(8), torch.zeros(8), 1e-6),                       # CPU tensors
        lambda: jg.layernorm_fwd(x, torch.zeros(7), torch.zeros(8), 1e-6),
        lambda: jg.layernorm_fwd(x.t(), torch.zeros(4), torch.zeros(4), 1e-6),
        lambda: jg.layernorm_fwd(x.double(), torch.zeros(8), torch.zeros(8), 1e-6),
        lambda: jg.layernorm_fwd(torch.tensor(1.0), f[:1], f[:1], 1e-6),
        lambda: jg.layernorm_bwd(torch.tensor(1.0), torch.tensor(1.0), f[:1], f[:1], f[:1]),
        lambda: jg.layernorm_bwd(x, x, torch.zeros(8), f, torch.zeros(5)),
        lambda: jg.linear_ce_fwd(x, W.half(), None, lab),
        lambda: jg.linear_ce_fwd(x, torch.zeros(6, 9), None, lab),
        lambda: jg.linear_ce_fwd(x, W, torch.zeros(5), lab),
        lambda: jg.linear_ce_fwd(x, W, None, lab.float()),
        lambda: jg.linear_ce_fwd(x, W, None, lab[:3]),
        lambda: jg.linear_ce_bwd(f, x, W, None, lab, torch.zeros(3)),
        lambda: jg.gated_ffn_fwd(x, W, torch.zeros(5, 8)),
        lambda: jg.gated_ffn_fwd(x, W, W, act="relu"),
        lambda: jg.gated_ffn_bwd(torch.zeros(4, 5), x, W, W),
        lambda: jg.linear_bwd(torch.zeros(4, 5), x, W),
        lambda: jg.linear_bwd(torch.zeros(4, 6), torch.zeros(8), W),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
