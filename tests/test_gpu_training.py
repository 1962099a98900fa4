"""The training operators on the GPU against the float64 oracle, element by
element, within bounds that follow from rounding (training_bounds.py)."""
import numpy as np
import pytest
import torch

import oracle
import training_bounds as tb
from oracle import training as ot

pytestmark = pytest.mark.gpu

TD = tb.TD


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


def _key(*parts):
    return sum((i + 1) * (sum(map(ord, p)) if isinstance(p, str) else int(p * 7)) for i, p in enumerate(parts))


def _dev(a, dtype="f32", shift=0):
    """The array on the GPU in dtype, starting `shift` elements into its buffer,
    and the rounded values back in float64."""
    t = torch.from_numpy(np.array(a, np.float32)).to(TD[dtype])
    buf = torch.empty(t.numel() + shift, dtype=TD[dtype], device="cuda")
    v = buf[shift:].view(t.shape)
    v.copy_(t)
    return v, t.double().numpy()


def _np(t):
    return t.double().cpu().numpy()


# ----------------------------------------------------------------------------- layer norm
LN_TYPES = [("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")]
LN_SHAPES = [(1, 1, 0), (3, 7, 0), (5, 64, 0), (37, 777, 0), (2, 256, 0), (130, 1000, 0), (70, 1024, 0), (9, 1025, 0),
             (6, 1536, 0), (4, 2050, 0), (3, 4096, 0), (2, 8192, 0), (3, 8193, 0), (3000, 136, 0), (16, 512, 1),
             (5, 1664, 1), (1, 1, 0), (3, 100003, 0), (2, 1 << 20, 0)]


def _depth(dim):
    """Additions on the longest path of a row sum: 32 in a thread, 5 + 8 joins; wider rows 1/256 of the row."""
    return max(64, dim / 256 + 32)


@pytest.mark.parametrize("xt,yt", LN_TYPES)
@pytest.mark.parametrize("rows,dim,shift", LN_SHAPES)
def test_layernorm_fwd(jg, rows, dim, shift, xt, yt):
    rng = np.random.default_rng(_key(rows, dim, xt, yt))
    x, xv = _dev(rng.standard_normal((rows, dim)) * 2 + rng.standard_normal((rows, 1)) * 3, xt, shift)
    w, wv = _dev(1 + 0.3 * rng.standard_normal(dim), shift=shift)
    b, bv = _dev(rng.standard_normal(dim), shift=shift)
    eps = 1e-6
    y, mean, rstd = jg.layernorm_fwd(x, w, b, eps, out_dtype=TD[yt])
    assert y.dtype == TD[yt] and mean.dtype == rstd.dtype == torch.float32
    mu, rs = ot.layer_norm_stats(xv, eps)
    ref = oracle.layer_norm(xv, wv, bv, eps)
    U, dep = tb.U, _depth(dim)
    emu = dep * U * np.abs(xv).mean(1) + U * np.abs(mu)
    d = np.abs(xv - mu[:, None])
    ed = emu[:, None] + U * d
    var = (d * d).mean(1)
    evar = (2 * d * ed + ed * ed).mean(1) + (dep + 2) * U * var
    lo = np.maximum(var + np.float64(np.float32(eps)) - evar, 1e-7)
    ers = 0.5 * evar / lo ** 1.5 + 6 * U * rs + 1e-7 * rs * eps / (var + eps)
    tb.check(_np(mean), mu, emu, "mean")
    tb.check(_np(rstd), rs, ers, "rstd")
    err = np.abs(wv) * (d * ers[:, None] + (rs + ers)[:, None] * ed) + 4 * U * (np.abs(ref) + np.abs(bv) + np.abs(wv) * d * rs[:, None])
    tb.check(_np(y), ref, tb.rounded(ref, err, yt), "y")


@pytest.mark.parametrize("xt,yt", LN_TYPES)
@pytest.mark.parametrize("rows,dim,shift", LN_SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_layernorm_bwd(jg, rows, dim, shift, xt, yt, res):
    rng = np.random.default_rng(_key(rows, dim, xt, yt, int(res)))
    x, xv = _dev(rng.standard_normal((rows, dim)) * 2 + rng.standard_normal((rows, 1)), xt, shift)
    dy, dyv = _dev(rng.standard_normal((rows, dim)), yt, shift)
    w, wv = _dev(1 + 0.3 * rng.standard_normal(dim), shift=shift)
    r, rv = _dev(rng.standard_normal((rows, dim)), xt, shift) if res else (None, None)
    mean, mv = _dev(xv.mean(1))
    rstd, sv = _dev(1 / np.sqrt(xv.var(1) + 1e-6))
    dx, dw, db = jg.layernorm_bwd(dy, x, w, mean, rstd, residual=r)
    rx, rw, rb = ot.layer_norm_bwd(dyv, xv, wv, mv, sv, rv)
    U, dep = tb.U, _depth(dim)
    xh, c = np.abs((xv - mv[:, None]) * sv[:, None]), np.abs(dyv * wv)
    m0, m1 = c.mean(1, keepdims=True), (c * xh).mean(1, keepdims=True)
    err = sv[:, None] * (8 * U * (c + m0 + xh * m1) + (dep + 4) * U * (m0 + xh * m1))
    if res:
        err = err + 2 * U * (np.abs(rv) + np.abs(rx))
    tb.check(_np(dx), rx, tb.rounded(rx, err, xt), "dx")
    n = rows + 16
    tb.check(_np(dw), rw, (n + 4) * U * np.abs(dyv * xh).sum(0), "dw")
    tb.check(_np(db), rb, n * U * np.abs(dyv).sum(0), "db")


def test_layernorm_leading_dims_needs_and_no_rows(jg):
    x = torch.randn(2, 3, 96, device="cuda")
    w, b = torch.randn(96, device="cuda"), torch.randn(96, device="cuda")
    y, mean, rstd = jg.layernorm_fwd(x, w, b, 1e-6)
    assert y.shape == x.shape and mean.shape == (2, 3)
    flat, m2, r2 = jg.layernorm_fwd(x.view(6, 96), w, b, 1e-6)
    assert torch.equal(flat.view_as(y), y) and torch.equal(m2, mean.view(-1)) and torch.equal(r2, rstd.view(-1))
    dy = torch.randn_like(x)
    full = jg.layernorm_bwd(dy, x, w, mean, rstd)
    dx, dw, db = jg.layernorm_bwd(dy, x, w, mean, rstd, needs=(False, True))
    assert dw is None and torch.equal(dx, full[0]) and torch.equal(db, full[2])
    e = torch.empty(0, 96, device="cuda")
    s = torch.empty(0, device="cuda")
    assert jg.layernorm_fwd(e, w, b, 1e-6)[0].shape == (0, 96)
    dx, dw, db = jg.layernorm_bwd(e, e, w, s, s)
    assert dx.shape == (0, 96) and not dw.any() and not db.any()


def test_layernorm_nan_row_stays_in_its_row(jg):
    """A row of NaN and one of infinities do not reach other rows' y or dx."""
    for dim in (129, 1024, 2048, 9000):
        x = torch.randn(7, dim, device="cuda")
        x[2], x[4, 0] = float("nan"), float("inf")
        w, b = torch.ones(dim, device="cuda"), torch.zeros(dim, device="cuda")
        y, mean, rstd = jg.layernorm_fwd(x, w, b, 1e-6)
        ok = [0, 1, 3, 5, 6]
        assert torch.isfinite(y[ok]).all() and torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
        dx = jg.layernorm_bwd(torch.randn_like(x), x, w, mean, rstd)[0]
        assert torch.isfinite(dx[ok]).all() and torch.isnan(dx[2]).all()


# ----------------------------------------------------------------------------- softmax cross entropy
CE_SHAPES = [(1, 8, 1, 0), (1, 64, 2, 0), (8, 1024, 174, 0), (129, 72, 257, 0), (300, 768, 1000, 0), (257, 65, 513, 0),
             (64, 128, 4097, 0), (33, 40, 30, 1), (600, 64, 300, 0), (5, 8, 9000, 0), (16, 200, 5000, 0), (9, 1032, 40, 0),
             (17, 512, 300, 0), (2600, 64, 300, 0), (700, 1100, 400, 0), (1, 1, 1, 0), (20, 1, 3, 0)]


def _ce_case(M, D, V, dtype, shift, key, ignore=0.2):
    rng = np.random.default_rng(_key(M, D, V, dtype, key))
    x, xv = _dev(rng.standard_normal((M, D)), dtype, shift)
    W, Wv = _dev(rng.standard_normal((V, D)) * 3 / np.sqrt(D), dtype, shift)
    b, bv = _dev(rng.standard_normal(V))
    lab = rng.integers(0, V, M)
    lab[rng.random(M) < ignore] = -100
    lab[0] = V - 1
    return rng, x, xv, W, Wv, b, bv, lab, torch.from_numpy(lab).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,D,V,shift", CE_SHAPES)
@pytest.mark.parametrize("smooth,bias", [(0.0, True), (0.1, True), (0.0, False)])
def test_linear_ce_fwd(jg, M, D, V, shift, dtype, smooth, bias):
    _, x, xv, W, Wv, b, bv, lab, labels = _ce_case(M, D, V, dtype, shift, 1)
    b, bv = (b, bv) if bias else (None, None)
    loss, lse = jg.linear_ce_fwd(x, W, b, labels, smoothing=smooth)
    rl, rs, z = ot.linear_ce(xv, Wv, bv, lab, smoothing=smooth)
    el, es = tb.ce_forward(xv, Wv, bv, z, rs, rl, lab, smooth)
    tb.check(_np(lse), rs, es, "lse")
    tb.check(_np(loss), rl, el, "loss")
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,D,V,shift", CE_SHAPES)
@pytest.mark.parametrize("smooth,bias,scale", [(0.0, True, 1e-3), (0.1, True, 64.0), (0.0, False, 1.0)])
def test_linear_ce_bwd(jg, M, D, V, shift, dtype, smooth, bias, scale):
    rng, x, xv, W, Wv, b, bv, lab, labels = _ce_case(M, D, V, dtype, shift, 2)
    b, bv = (b, bv) if bias else (None, None)
    dl, dlv = _dev(rng.standard_normal(M) * scale)
    _, rs, z = ot.linear_ce(xv, Wv, bv, lab, smoothing=smooth)
    lse, lsev = _dev(rs)
    dx, dW, db = jg.linear_ce_bwd(dl, x, W, b, labels, lse, smoothing=smooth)
    dz = ot.linear_ce_dz(z, lsev, dlv, lab, smoothing=smooth)
    e = tb.ce_dz(xv, Wv, bv, z, lsev, dlv, lab, smooth, dtype)
    e[lab == -100] = 0
    tb.check(_np(db), dz.sum(0), e.sum(0) + 2 * tb.U * (M + 16) * np.abs(dz).sum(0), "dbias")
    # the 16-bit dz: half a step of itself, or of the smallest normal of the scaled type
    h = 0 if dtype == "f32" else tb.HALF[dtype]
    floor = 2.0 ** -38 * np.abs(dlv).max() if dtype == "f16" else 0.0
    er = e + h * (np.abs(dz) + e) + floor * (lab != -100)[:, None]
    rx, rw = dz @ Wv, dz.T @ xv
    tb.check(_np(dx), rx, tb.rounded(rx, tb.product(dz, Wv.T, er), dtype), "dx")
    tb.check(_np(dW), rw, tb.rounded(rw, tb.product(dz.T, xv.T, er.T), dtype), "dW")
    jg.ops_sync()


def _sample(rng, n, k, tile=256):
    """k of n places, with those at both ends and around tiles' borders."""
    edge = [i for b in (0, tile, n // 2 // tile * tile, n) for i in (b - 1, b) if 0 <= i < n]
    return np.unique(np.concatenate([edge, rng.integers(0, n, k)]).astype(int))


@pytest.mark.parametrize("dtype,M,D,V", [("bf16", 2048, 64, 40000), ("f32", 2048, 40, 40001), ("f16", 700, 33, 150001)])
def test_linear_ce_fwd_many_tiles(jg, dtype, M, D, V):
    """Row statistics carried over several column tiles."""
    rng, x, xv, W, Wv, b, bv, lab, labels = _ce_case(M, D, V, dtype, 0, 6)
    loss, lse = jg.linear_ce_fwd(x, W, b, labels, smoothing=0.1)
    r = _sample(rng, M, 24)
    rl, rs, z = ot.linear_ce(xv[r], Wv, bv, lab[r], smoothing=0.1)
    el, es = tb.ce_forward(xv[r], Wv, bv, z, rs, rl, lab[r], 0.1)
    tb.check(_np(lse)[r], rs, es, "lse")
    tb.check(_np(loss)[r], rl, el, "loss")
    # every row against float64 on the device; the rows' bounds are of one size, 4 is for their spread
    z64 = x.double() @ W.double().T + b.double()
    assert (lse.double() - torch.logsumexp(z64, 1)).abs().max() <= 4 * es.max()
    jg.ops_sync()


@pytest.mark.parametrize("dtype,M,D,V", [("bf16", 20000, 64, 9000), ("f16", 20001, 72, 9001), ("f32", 12000, 64, 5000),
                                         ("f32", 12001, 30, 9001)])
def test_linear_ce_bwd_in_pieces(jg, dtype, M, D, V):
    """Vocabularies whose dz does not fit the workspace's 256 MB at once."""
    rng, x, xv, W, Wv, b, bv, lab, labels = _ce_case(M, D, V, dtype, 0, 7)
    smooth = 0.1
    dl, dlv = _dev(rng.standard_normal(M) / M)
    # in blocks of rows: 64-bit lse, then dz as the oracle's, on the device
    x64, W64, b64 = x.double(), W.double(), b.double()
    lse = torch.cat([torch.logsumexp(x64[i:i + 4000] @ W64.T + b64, 1) for i in range(0, M, 4000)]).float()
    lsev = _np(lse)
    dx, dW, db = jg.linear_ce_bwd(dl, x, W, b, labels, lse, smoothing=smooth)
    h = 0 if dtype == "f32" else tb.HALF[dtype]
    floor = 2.0 ** -38 * np.abs(dlv).max() if dtype == "f16" else 0.0

    def dz_of(rows, classes):
        z = xv[rows] @ Wv[classes].T + bv[classes]
        keep = (lab[rows] != -100)[:, None]
        hit = np.arange(V)[classes][None] == lab[rows][:, None]
        g = dlv[rows][:, None] * keep
        dz = g * (np.exp(z - lsev[rows][:, None]) - smooth / V - (1 - smooth) * hit)
        e = tb.ce_logits(xv[rows], Wv[classes], bv[classes])
        arg = e + 4 * tb.U * (np.abs(z) + np.abs(lsev[rows])[:, None] + 4)
        p = np.exp(z - lsev[rows][:, None])
        e = np.abs(g) * (p * np.expm1(arg) + 2 * tb.U + 6 * tb.U * (p + hit + smooth))
        return dz, e, e + h * (np.abs(dz) + e) + floor * keep
    r, c = _sample(rng, M, 40), _sample(rng, V, 40)
    every = slice(None)
    dz, _, er = dz_of(r, every)
    rx = dz @ Wv
    tb.check(_np(dx)[r], rx, tb.rounded(rx, tb.product(dz, Wv.T, er), dtype), "dx")
    dz, e, er = dz_of(every, c)
    rw = dz.T @ xv
    tb.check(_np(dW)[c], rw, tb.rounded(rw, tb.product(dz.T, xv.T, er.T), dtype), "dW")
    tb.check(_np(db)[c], dz.sum(0), e.sum(0) + 2 * tb.U * (M + 16) * np.abs(dz).sum(0), "dbias")
    # one gradient at a time gives the same
    assert torch.equal(jg.linear_ce_bwd(dl, x, W, b, labels, lse, smoothing=smooth, needs=(True, False, False))[0], dx)
    assert torch.equal(jg.linear_ce_bwd(dl, x, W, b, labels, lse, smoothing=smooth, needs=(False, True, False))[1], dW)
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_linear_ce_dloss_of_rows_without_a_gradient(jg, dtype):
    """dloss of ignored rows is not used: not its size, not an infinity, not NaN."""
    M, D, V = 150, 64, 300
    _, x, _, W, _, b, _, lab, labels = _ce_case(M, D, V, dtype, 0, 8, ignore=0.5)
    _, lse = jg.linear_ce_fwd(x, W, b, labels)
    dl = torch.randn(M, device="cuda")
    want = jg.linear_ce_bwd(torch.where(labels == -100, 0.0, dl), x, W, b, labels, lse)
    for v in (1e30, float("inf"), float("nan")):
        got = jg.linear_ce_bwd(torch.where(labels == -100, v, dl), x, W, b, labels, lse)
        for a, r in zip(got, want):
            assert torch.equal(a, r), v


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("smooth", [0.75, 0.8, 0.97])
def test_linear_ce_strong_smoothing(jg, dtype, smooth):
    """Certain of a wrong class: the 16-bit dz is largest, 1 / (1 - smoothing) in its unit."""
    M, D, V = 150, 64, 300
    rng, x, xv, _, Wv, b, bv, lab, labels = _ce_case(M, D, V, dtype, 0, 10)
    W, Wv = _dev(8 * Wv, dtype)
    dl, dlv = _dev(rng.standard_normal(M))
    _, rs, z = ot.linear_ce(xv, Wv, bv, lab, smoothing=smooth)
    assert (np.exp(z - rs[:, None]).max(1) > 0.999).any()
    lse, lsev = _dev(rs)
    dx, dW, db = jg.linear_ce_bwd(dl, x, W, b, labels, lse, smoothing=smooth)
    dz = ot.linear_ce_dz(z, lsev, dlv, lab, smoothing=smooth)
    e = tb.ce_dz(xv, Wv, bv, z, lsev, dlv, lab, smooth, dtype)
    e[lab == -100] = 0
    tb.check(_np(db), dz.sum(0), e.sum(0) + 2 * tb.U * (M + 16) * np.abs(dz).sum(0), "dbias")
    # fp16: half its smallest subnormal, 2^-25, in units of max |dloss| (1 - smoothing) / 2^(14 + floor(log2(1 - smoothing)))
    h = 0 if dtype == "f32" else tb.HALF[dtype]
    floor = 2.0 ** -38 * np.abs(dlv).max() if dtype == "f16" else 0.0
    er = e + h * (np.abs(dz) + e) + floor * (lab != -100)[:, None]
    rx, rw = dz @ Wv, dz.T @ xv
    tb.check(_np(dx), rx, tb.rounded(rx, tb.product(dz, Wv.T, er), dtype), "dx")
    tb.check(_np(dW), rw, tb.rounded(rw, tb.product(dz.T, xv.T, er.T), dtype), "dW")


def test_linear_ce_forms_of_labels_and_dloss(jg):
    """int32 labels, one dloss as a number or as a tensor without dimensions."""
    _, x, _, W, _, b, _, lab, labels = _ce_case(200, 64, 300, "bf16", 0, 9)
    loss, lse = jg.linear_ce_fwd(x, W, b, labels)
    l32, s32 = jg.linear_ce_fwd(x, W, b, labels.int())
    assert torch.equal(loss, l32) and torch.equal(lse, s32)
    want = jg.linear_ce_bwd(torch.full((200,), 0.25, device="cuda"), x, W, b, labels, lse)
    for dl in (0.25, torch.tensor(0.25), torch.tensor(0.25, device="cuda", dtype=torch.float64)):
        for a, r in zip(jg.linear_ce_bwd(dl, x, W, b, labels.int(), lse), want):
            assert torch.equal(a, r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 33])
def test_linear_ce_rows_without_a_label(jg, dtype, D):
    """Every row ignored: loss 0, gradients 0, lse still the row's own.  Bad
    labels: loss NaN, no gradient, reported once."""
    from video_vit_encoder_gb300._lib import ERR_ARG, JepaError
    M, V = 140, 300
    _, x, xv, W, Wv, b, bv, lab, _ = _ce_case(M, D, V, dtype, 0, 3)
    none = torch.full((M,), 7, device="cuda")
    loss, lse = jg.linear_ce_fwd(x, W, b, none, ignore_index=7)
    assert not loss.any()
    rs = ot.linear_ce(xv, Wv, bv, lab)[1]
    assert np.abs(_np(lse) - rs).max() < 1e-3
    for g in jg.linear_ce_bwd(1.0, x, W, b, none, lse, ignore_index=7):
        assert not g.any()
    jg.ops_sync()
    bad = torch.full((M,), -100, device="cuda")
    bad[3], bad[5], bad[8] = V, -1, (1 << 32) + 2
    loss, lse = jg.linear_ce_fwd(x, W, b, bad)
    assert torch.isnan(loss[[3, 5, 8]]).all() and not loss[[0, 1, 2, 4, 6]].any()
    with pytest.raises(JepaError) as e:
        jg.ops_sync()
    assert e.value.status == ERR_ARG
    for g in jg.linear_ce_bwd(1.0, x, W, b, bad, lse):
        assert not g.any()
    with pytest.raises(JepaError):
        jg.ops_sync()
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 33])
def test_linear_ce_masked_classes(jg, dtype, D):
    """A bias of -inf, and one of the lowest float, take classes out: a run of
    600 (whole tiles), and all but one."""
    M, V = 70, 1030
    _, x, xv, W, Wv, b, bv, lab, _ = _ce_case(M, D, V, dtype, 0, 4)
    lab[:] = 3
    for mask in (slice(200, 800), np.r_[0:3, 4:V]):
        for low in (-np.inf, np.finfo(np.float32).min):
            bb = bv.copy()
            bb[mask] = low
            bt, _ = _dev(bb)
            labels = torch.from_numpy(lab).cuda()
            loss, lse = jg.linear_ce_fwd(x, W, bt, labels)
            with np.errstate(over="ignore"):
                rl, rs, z = ot.linear_ce(xv, Wv, bb, lab)
            keep = np.setdiff1d(np.arange(V), np.arange(V)[mask])
            el, es = tb.ce_forward(xv, Wv[keep], bb[keep], z[:, keep], rs, rl, np.zeros(M, int), 0.0)
            el = el + tb.ce_logits(xv, Wv, bv)[:, 3]
            tb.check(_np(lse), rs, es + 1e-30, "lse")
            tb.check(_np(loss), rl, el + es + 2e-6, "loss")
            dx, dW, db = jg.linear_ce_bwd(1.0, x, W, bt, labels, lse)
            assert not dW[mask].any() and not db[mask].any()
            assert torch.isfinite(dx).all() and torch.isfinite(dW).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 33])
def test_linear_ce_nan_rows(jg, dtype, D):
    """A NaN in a row's x makes that row's loss NaN and no other's; every class
    masked out gives the formula's NaN loss."""
    M, V = 140, 700
    _, x, _, W, _, b, _, lab, labels = _ce_case(M, D, V, dtype, 0, 5, ignore=0.0)
    x = x.clone()
    x[17, 3] = float("nan")
    loss, lse = jg.linear_ce_fwd(x, W, b, labels)
    assert torch.isnan(loss[17]) and torch.isnan(lse[17])
    keep = torch.arange(M, device="cuda") != 17
    assert torch.isfinite(loss[keep]).all()
    loss, lse = jg.linear_ce_fwd(x, W, torch.full_like(b, float("-inf")), labels)
    assert (lse[keep] == float("-inf")).all() and torch.isnan(loss).all()


# ----------------------------------------------------------------------------- gated feed-forward
FFN_SHAPES = [(1, 64, 8, 0), (1, 8, 1, 0), (8, 1024, 256, 0), (129, 72, 136, 0), (300, 256, 520, 0), (257, 128, 1000, 0),
              (5, 33, 17, 0), (200, 65, 300, 0), (40, 64, 64, 1), (700, 128, 256, 0), (16, 200, 72, 0), (12, 1032, 520, 0),
              (17, 512, 77, 0), (2, 4, 3, 0), (2600, 72, 136, 0), (400, 1100, 520, 0), (1, 1, 1, 0),
              (20, 1, 3, 0)]


def _ffn_case(M, D, F, dtype, shift, bias, key):
    rng = np.random.default_rng(_key(M, D, F, dtype, key))
    x, xv = _dev(rng.standard_normal((M, D)) * 1.5, dtype, shift)
    Wg, Wgv = _dev(rng.standard_normal((F, D)) / np.sqrt(D), dtype, shift)
    Wu, Wuv = _dev(rng.standard_normal((F, D)) / np.sqrt(D), dtype, shift)
    bg, bgv = _dev(rng.standard_normal(F)) if bias else (None, None)
    bu, buv = _dev(rng.standard_normal(F)) if bias else (None, None)
    g, u = ot.gated_project(xv, Wgv, Wuv, bgv, buv)
    eg, eu = tb.product(xv, Wgv) + 2 * tb.U * np.abs(g), tb.product(xv, Wuv) + 2 * tb.U * np.abs(u)
    return rng, (x, Wg, Wu, bg, bu), (xv, Wgv, Wuv, bgv, buv), g, u, eg, eu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,D,F,shift", FFN_SHAPES)
@pytest.mark.parametrize("act,bias", [("silu", False), ("gelu", True)])
def test_gated_ffn_fwd(jg, M, D, F, shift, dtype, act, bias):
    _, t, v, g, u, eg, eu = _ffn_case(M, D, F, dtype, shift, bias, 1)
    h = jg.gated_ffn_fwd(*t, act=act)
    ref = ot.gate_act(g, act) * u
    ea, _ = tb.gate(g, u, eg, eu, act)
    err = ea * (np.abs(u) + eu) + np.abs(ot.gate_act(g, act)) * eu + 4 * tb.U * np.abs(ref)
    tb.check(_np(h), ref, tb.rounded(ref, err, dtype), "h")
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,D,F,shift", FFN_SHAPES)
@pytest.mark.parametrize("act,bias", [("silu", True), ("gelu", True), ("silu", False)])
def test_gated_ffn_bwd(jg, M, D, F, shift, dtype, act, bias):
    rng, t, v, g, u, eg, eu = _ffn_case(M, D, F, dtype, shift, bias, 2)
    dh, dhv = _dev(rng.standard_normal((M, F)), dtype, shift)
    dx, dwg, dwu, dbg, dbu = jg.gated_ffn_bwd(dh, *t, act=act)
    a, da = ot.gate_act(g, act), ot.gate_act_grad(g, act)
    ea, ed = tb.gate(g, u, eg, eu, act)
    dg, du = dhv * u * da, dhv * a
    edg = np.abs(dhv) * (eu * (np.abs(da) + ed) + np.abs(u) * ed) + 6 * tb.U * np.abs(dg)
    edu = np.abs(dhv) * ea + 4 * tb.U * np.abs(du)
    tb.check(_np(dbg), dg.sum(0), edg.sum(0) + 2 * tb.U * (M + 16) * np.abs(dg).sum(0), "dbg")
    tb.check(_np(dbu), du.sum(0), edu.sum(0) + 2 * tb.U * (M + 16) * np.abs(du).sum(0), "dbu")
    if dtype != "f32":
        edg, edu = tb.rounded(dg, edg, dtype), tb.rounded(du, edu, dtype)
    xv, Wgv, Wuv = v[:3]
    rx = dg @ Wgv + du @ Wuv
    # one sum over both halves: 2F terms
    ex = tb.product(np.concatenate([dg, du], 1), np.concatenate([Wgv, Wuv]).T, np.concatenate([edg, edu], 1))
    tb.check(_np(dx), rx, tb.rounded(rx, ex, dtype), "dx")
    for got, d, ee, what in ((dwg, dg, edg, "dWg"), (dwu, du, edu, "dWu")):
        ref = d.T @ xv
        tb.check(_np(got), ref, tb.rounded(ref, tb.product(d.T, xv.T, ee.T), dtype), what)
    jg.ops_sync()


def test_gated_ffn_large_gates(jg):
    """Gates far out on both sides: silu and gelu saturate, nothing overflows."""
    M, F = 150, 200
    for D in (64, 63):
        for dtype in ("bf16", "f32"):
            x, _ = _dev(np.ones((M, D)), dtype)
            Wg, _ = _dev(np.where(np.arange(F)[:, None] % 2 == 0, 4.0, -4.0) * np.ones((1, D)), dtype)
            Wu, _ = _dev(np.ones((F, D)) / 8, dtype)
            dh, _ = _dev(np.ones((M, F)), dtype)
            for act in ("silu", "gelu"):
                h = _np(jg.gated_ffn_fwd(x, Wg, Wu, act=act))
                u, g = D / 8, 4.0 * D
                assert np.all(np.abs(h[:, ::2] - g * u) <= g * u * 2 * tb.HALF[dtype] + 1e-3) and not h[:, 1::2].any()
                for t in jg.gated_ffn_bwd(dh, x, Wg, Wu, act=act)[:3]:
                    assert torch.isfinite(t).all()
    jg.ops_sync()


# ----------------------------------------------------------------------------- linear layer
LIN_SHAPES = [(1, 1, 1, 0), (1, 64, 64, 0), (8, 174, 1024, 0), (129, 136, 72, 0), (300, 520, 256, 0), (257, 33, 65, 0),
              (1000, 256, 128, 0), (40, 64, 64, 1), (2305, 136, 72, 0), (3, 1000, 2048, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,shift", LIN_SHAPES)
def test_linear_bwd(jg, M, N, K, shift, dtype):
    rng = np.random.default_rng(_key(M, N, K, dtype))
    A, Av = _dev(rng.standard_normal((M, K)), dtype, shift)
    W, Wv = _dev(rng.standard_normal((N, K)), dtype, shift)
    d, dv = _dev(rng.standard_normal((M, N)), dtype, shift)
    dA, dW, db = jg.linear_bwd(d, A, W)
    rA, rW, rb = ot.linear_bwd(dv, Av, Wv)
    tb.check(_np(dA), rA, tb.rounded(rA, tb.product(dv, Wv.T), dtype), "dA")
    tb.check(_np(dW), rW, tb.rounded(rW, tb.product(dv.T, Av.T), dtype), "dW")
    tb.check(_np(db), rb, 2 * tb.U * (M + 16) * np.abs(dv).sum(0), "dbias")
    only = jg.linear_bwd(d, A, W, bias=False, needs=(False, True))
    assert only[0] is None and only[2] is None and torch.equal(only[1], dW)
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(jg, dtype):
    """No rows: empty outputs, zero weight gradients."""
    e = torch.empty(0, 64, dtype=TD[dtype], device="cuda")
    W = torch.randn(96, 64, device="cuda").to(TD[dtype])
    lab = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = jg.linear_ce_fwd(e, W, None, lab)
    assert loss.shape == (0,)
    dx, dW, db = jg.linear_ce_bwd(loss, e, W, None, lab, lse)
    assert dx.shape == (0, 64) and not dW.any() and not db.any()
    assert jg.gated_ffn_fwd(e, W, W).shape == (0, 96)
    dh = torch.empty(0, 96, dtype=TD[dtype], device="cuda")
    dx, *rest = jg.gated_ffn_bwd(dh, e, W, W)
    assert dx.shape == (0, 64) and not any(t.any() for t in rest)
    dA, dW, db = jg.linear_bwd(dh, e, W)
    assert dA.shape == (0, 64) and not dW.any() and not db.any()
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------- together
def _block(jg, p, x, labels, n):
    """One training step of a gated MLP block and classifier on fp32 rows x:
    x + down(gated(ln(x))) -> ln -> classifier -> mean loss, and all gradients."""
    y1, m1, r1 = jg.layernorm_fwd(x, p["w1"], p["b1"], 1e-6, out_dtype=p["Wg"].dtype)
    h = jg.gated_ffn_fwd(y1, p["Wg"], p["Wu"], p["bg"], p["bu"])
    x2 = jg.linear(h, p["Wd"], p["bd"], 2, out=x.clone())
    y2, m2, r2 = jg.layernorm_fwd(x2, p["w2"], p["b2"], 1e-6, out_dtype=p["Wg"].dtype)
    loss, lse = jg.linear_ce_fwd(y2, p["Wc"], p["bc"], labels)
    dy2, dWc, dbc = jg.linear_ce_bwd(1.0 / n, y2, p["Wc"], p["bc"], labels, lse)
    dx2, dw2, db2 = jg.layernorm_bwd(dy2, x2, p["w2"], m2, r2)
    dh, dWd, dbd = jg.linear_bwd(dx2.to(h.dtype), h, p["Wd"])
    dy1, dWg, dWu, dbg, dbu = jg.gated_ffn_bwd(dh, y1, p["Wg"], p["Wu"], p["bg"], p["bu"])
    dx, dw1, db1 = jg.layernorm_bwd(dy1, x, p["w1"], m1, r1, residual=dx2)
    return loss, dict(x=dx, w1=dw1, b1=db1, Wg=dWg, Wu=dWu, bg=dbg, bu=dbu, Wd=dWd, bd=dbd, w2=dw2, b2=db2, Wc=dWc,
                      bc=dbc)


def _block_params(rng, D, F, V, dtype):
    f = {"w1": 1 + 0.1 * rng.standard_normal(D), "b1": 0.1 * rng.standard_normal(D),
         "w2": 1 + 0.1 * rng.standard_normal(D), "b2": 0.1 * rng.standard_normal(D),
         "bg": 0.1 * rng.standard_normal(F), "bu": 0.1 * rng.standard_normal(F), "bd": 0.1 * rng.standard_normal(D),
         "bc": 0.1 * rng.standard_normal(V)}
    m = {"Wg": rng.standard_normal((F, D)) / np.sqrt(D), "Wu": rng.standard_normal((F, D)) / np.sqrt(D),
         "Wd": rng.standard_normal((D, F)) / np.sqrt(F), "Wc": 2 * rng.standard_normal((V, D)) / np.sqrt(D)}
    p, v = {}, {}
    for k, a in f.items():
        p[k], v[k] = _dev(a)
    for k, a in m.items():
        p[k], v[k] = _dev(a, dtype)
    return p, v


@pytest.mark.parametrize("dtype,tol", [("f32", 2e-5), ("bf16", 3e-2), ("f16", 4e-3)])
def test_training_step_against_autograd(jg, dtype, tol):
    """The operators run together as one training step, against float64 autograd
    of the same block.  Tolerance relative to each gradient's norm: eight
    roundings to the type on the longest path (y1, h, y2, dz, dy2, dx2, dh,
    dgate) of eps/2 each, sqrt(8) HALF = 0.011 (bf16) if they add as noise, and
    2.5 times that; fp32 accumulations over at most 512 terms for f32."""
    rng = np.random.default_rng(11)
    M, D, F, V = 300, 256, 512, 1000
    p, v = _block_params(rng, D, F, V, dtype)
    x, xv = _dev(rng.standard_normal((M, D)))
    lab = rng.integers(0, V, M)
    lab[::7] = -100
    n = int((lab >= 0).sum())
    loss, grads = _block(jg, p, x, torch.from_numpy(lab).cuda(), n)
    t = {k: torch.from_numpy(a).requires_grad_() for k, a in v.items()}
    tx = torch.from_numpy(xv).requires_grad_()
    F_ = torch.nn.functional
    y = F_.layer_norm(tx, (D,), t["w1"], t["b1"], 1e-6)
    h = F_.silu(y @ t["Wg"].T + t["bg"]) * (y @ t["Wu"].T + t["bu"])
    y2 = F_.layer_norm(tx + h @ t["Wd"].T + t["bd"], (D,), t["w2"], t["b2"], 1e-6)
    ref = F_.cross_entropy(y2 @ t["Wc"].T + t["bc"], torch.from_numpy(lab))
    ref.backward()
    assert abs(float(loss.double().sum()) / n - float(ref)) <= tol * max(1.0, float(ref))
    t["x"] = tx
    for k, g in grads.items():
        r = t[k].grad.numpy()
        assert np.linalg.norm(_np(g) - r) <= tol * np.linalg.norm(r), (k, np.linalg.norm(_np(g) - r) / np.linalg.norm(r))
    jg.ops_sync()


def test_training_step_in_a_graph(jg):
    """The step captured into two CUDA graphs that replay in turn and at once on
    two streams, with new inputs in place, gives the eager step's bits."""
    rng = np.random.default_rng(12)
    M, D, F, V = 300, 256, 512, 1000
    p, _ = _block_params(rng, D, F, V, "bf16")
    xs = [torch.randn(M, D, device="cuda") for _ in range(3)]
    labs = [torch.randint(0, V, (M,), device="cuda") for _ in range(3)]
    eager = [_block(jg, p, a, b, M) for a, b in zip(xs, labs)]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        sx, sl = xs[i].clone(), labs[i].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _block(jg, p, sx, sl, M)
        graphs.append((g, sx, sl, out))

    def same(out, ref):
        assert torch.equal(out[0], ref[0])
        for k in ref[1]:
            assert torch.equal(out[1][k], ref[1][k]), k
    for g, *_ in graphs:
        g.replay()
    torch.cuda.synchronize()
    same(graphs[0][3], eager[0])
    same(graphs[1][3], eager[1])
    graphs[0][1].copy_(xs[2])
    graphs[0][2].copy_(labs[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    same(graphs[0][3], eager[2])
    same(graphs[1][3], eager[1])
    jg.ops_sync()


def test_calls_on_two_streams(jg):
    """The same calls issued on two streams at once, by argument and by context,
    give the default stream's bits."""
    x = torch.randn(500, 512, device="cuda").bfloat16()
    W, W2 = (torch.randn(1200, 512, device="cuda") / 22).bfloat16(), (torch.randn(1200, 512, device="cuda") / 22).bfloat16()
    lab = torch.randint(0, 1200, (500,), device="cuda")
    dh = torch.randn(500, 1200, device="cuda").bfloat16()

    def step(stream=None):
        loss, lse = jg.linear_ce_fwd(x, W, None, lab, stream=stream)
        return (loss, lse) + jg.linear_ce_bwd(1.0, x, W, None, lab, lse, stream=stream) + \
            jg.gated_ffn_bwd(dh, x, W, W2, stream=stream)
    ref = step()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        outs.append(step(s1))
        with torch.cuda.stream(s2):
            outs.append(step())
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, ref):
            assert torch.equal(a, b)
    jg.ops_sync()


def test_inputs_dropped_while_another_stream_uses_them(jg):
    """Inputs that are dropped right after a call on another stream: their
    memory is not given out before that stream is done with it."""
    side = torch.cuda.Stream()
    W = (torch.randn(300, 256, device="cuda") / 16).bfloat16()
    lab = torch.randint(0, 300, (400,), device="cuda")
    x = torch.randn(400, 256, device="cuda").bfloat16()
    want = jg.linear_ce_fwd(x, W, None, lab)
    ref = jg.linear_ce_bwd(1.0, x, W, None, lab, want[1])
    keep = x.clone()
    torch.cuda.synchronize()
    for _ in range(3):
        x = keep.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)   # clocks, about 10 ms
        got = jg.linear_ce_bwd(1.0, x, W, None, lab, want[1], stream=side)
        del x
        others = [torch.zeros(400, 256, device="cuda", dtype=torch.bfloat16) for _ in range(8)]
        torch.cuda.synchronize()
        for a, r in zip(got, ref):
            assert torch.equal(a, r)
        del others


def test_offsets_past_32_bits_in_products(jg):
    """The same on the tensor-core path: a classifier whose W passes 2^31
    elements, a gate whose h does, a linear layer whose dout does."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, dim, M = (1 << 20) + 3, 2056, 40
    big = torch.randn(rows, dim, device="cuda", generator=g, dtype=torch.bfloat16)
    inp = (torch.randn(M, dim, device="cuda", generator=g) / 45).bfloat16()
    lab = torch.randint(0, rows, (M,), device="cuda", generator=g)
    lab[:3] = torch.tensor([rows - 1, rows - 2, 0])
    loss, lse = jg.linear_ce_fwd(inp, big, None, lab)
    z = torch.cat([inp.double() @ big[i:i + 65536].double().T for i in range(0, rows, 65536)], 1)
    ref = torch.logsumexp(z, 1)
    # 2056 products a logit, 2^-23 each at most, of logits of size 1
    assert (lse.double() - ref).abs().max() < 1e-4
    assert (loss.double() - (ref - z.gather(1, lab[:, None])[:, 0])).abs().max() < 2e-4
    dx, dW, db = jg.linear_ce_bwd(1.0, inp, big, None, lab, lse)
    tail = slice(rows - 5, rows)
    dz = torch.exp(z - ref[:, None])
    dz[torch.arange(M, device="cuda"), lab] -= 1
    # dz and the results are rounded to bf16, half a step each
    want = dz[:, tail].T @ inp.double()
    assert (dW[tail].double() - want).abs().max() <= 2 ** -7 * want.abs().max()
    want = sum(dz[:, i:i + 65536] @ big[i:i + 65536].double() for i in range(0, rows, 65536))
    assert (dx.double() - want).norm() <= 2 ** -7 * want.norm()
    del z, dz, dW
    # dout = big, K = 8
    A = torch.randn(rows, 8, device="cuda", generator=g).bfloat16()
    W = torch.randn(dim, 8, device="cuda", generator=g).bfloat16()
    dA, dW, db = jg.linear_bwd(big, A, W)
    want = big[tail].double() @ W.double()
    assert (dA[tail].double() - want).norm() <= 2 ** -7 * want.norm()
    want = sum(big[i:i + 65536].double().T @ A[i:i + 65536].double() for i in range(0, rows, 65536))
    assert (dW.double() - want).norm() <= 2 ** -7 * want.norm()
    want = sum(big[i:i + 65536].double().sum(0) for i in range(0, rows, 65536))
    assert (db.double() - want).abs().max() <= 2 * tb.U * rows * 0.8 * 16   # of sums of |dout| of 0.8 a row
    # h and dh [rows, dim], D = 8
    h = jg.gated_ffn_fwd(A, W, W)
    gt = A[tail].double() @ W.double().T
    want = gt * torch.sigmoid(gt) * gt
    assert (h[tail].double() - want).norm() <= 2 ** -7 * want.norm()
    dx, dWg, *_ = jg.gated_ffn_bwd(big, A, W, W)
    s = torch.sigmoid(gt)
    dh = big[tail].double()
    want = (dh * gt * s * (1 + gt * (1 - s))) @ W.double() + (dh * gt * s) @ W.double()
    assert (dx[tail].double() - want).norm() <= 2 ** -6 * want.norm()
    jg.ops_sync()


def test_offsets_past_32_bits(jg):
    """Rows and classes whose element offset passes 2^31: the last ones are
    right, in every operator that walks such a matrix."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rows, dim = (1 << 20) + 3, 2056      # 2.16e9 elements
    x = torch.randn(rows, dim, device="cuda", generator=g, dtype=torch.bfloat16)
    w, b = torch.randn(dim, device="cuda", generator=g), torch.randn(dim, device="cuda", generator=g)
    y, mean, rstd = jg.layernorm_fwd(x, w, b, 1e-6)
    tail = slice(rows - 5, rows)
    yt, mt, rt = jg.layernorm_fwd(x[tail], w, b, 1e-6)
    assert torch.equal(y[tail], yt) and torch.equal(mean[tail], mt) and torch.equal(rstd[tail], rt)
    dx, _, _ = jg.layernorm_bwd(y, x, w, mean, rstd)
    assert torch.equal(dx[tail], jg.layernorm_bwd(y[tail], x[tail], w, mt, rt)[0])
    del y, dx
    # x as the weights of a classifier of `rows` classes, a few rows of input
    M = 6
    inp = (torch.randn(M, dim, device="cuda", generator=g) / 45).bfloat16()
    lab = torch.tensor([rows - 1, 0, rows - 2, -100, rows - 3, 5], device="cuda")
    loss, lse = jg.linear_ce_fwd(inp, x, None, lab)
    z = torch.cat([inp.double() @ x[i:i + 65536].double().T for i in range(0, rows, 65536)], 1)
    ref = torch.logsumexp(z, 1)
    assert (lse.double() - ref).abs().max() < 1e-4
    keep = [0, 1, 2, 4, 5]
    assert (loss.double()[keep] - (ref - z.gather(1, lab.clamp(min=0)[:, None])[:, 0])[keep]).abs().max() < 1e-4
    _, dW, db = jg.linear_ce_bwd(1.0, inp, x, None, lab, lse, needs=(False, True, True))
    dz = torch.exp(z[:, tail] - ref[:, None])
    for i, l in ((0, rows - 1), (2, rows - 2), (4, rows - 3)):
        dz[i, l - (rows - 5)] -= 1
    dz[3] = 0
    want = dz.T @ inp.double()
    assert (dW[tail].double() - want).abs().max() <= 2 ** -7 * want.abs().max()
    assert (db[tail].double() - dz.sum(0)).abs().max() < 1e-5
    jg.ops_sync()
