"""Products over very long sums.  The tensor core truncates its accumulator; a
step of 16 products of one sign costs the sum up to 2^-23 of itself (measured
0.85 of that for long sums, and n + 2 units at most after n < 40 steps), so a sum
with a 16-bit result stays in it for at most LONG steps, which cost half as much
as the result's rounding: 2^11 * 2^-23 = HALF / 2 in fp16, 2^14 * 2^-23 = HALF /
2 in bf16.  Results held in fp32 (lse, loss) take 32 steps in one go, SHORT.
What is added in fp32 after that is rounded."""
import numpy as np
import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu

LONG = {"f16": 2.0 ** -12, "bf16": 2.0 ** -9}
PIECE = {"f16": 1 << 15, "bf16": 1 << 18}   # products in LONG steps
SHORT = 34 * 2.0 ** -23


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


def _positive(g, rows, cols, scale, dtype):
    """Values in [scale / 4, scale], columns of different size."""
    t = torch.rand(rows, cols, device="cuda", generator=g, dtype=torch.float32).mul_(0.5).add_(0.5)
    t.mul_((0.5 + 0.5 * torch.rand(cols, device="cuda", generator=g)) * scale)
    return t.to(tb.TD[dtype])


def _blocks(rows, step=1 << 20):
    return [slice(i, min(i + step, rows)) for i in range(0, rows, step)]


def _relative(got, want, dtype, terms, extra=0.0, n=None):
    """Every entry within a rounding of the type and the loss; the mean error,
    in which the roundings of n entries cancel (uniform, so a standard deviation
    of HALF / sqrt 3; six of them), within the loss."""
    e = (got.double() - want) / want
    fp32 = LONG[dtype] + (terms / PIECE[dtype] + 32) * tb.U + extra
    half = tb.HALF[dtype]
    assert e.abs().max() <= half + fp32, e.abs().max()
    assert e.mean().abs() <= fp32 + 6 * half / np.sqrt(3 * (n or e.numel())), e.mean()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linear_bwd_over_many_rows(jg, dtype):
    """dW over 2^24 rows; the sums are rounded to fp32 from piece to piece."""
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = 1 << 24, 64, 64
    d, A = _positive(g, M, N, 1 / 32, dtype), _positive(g, M, K, 1 / 32, dtype)
    W = torch.zeros(N, K, device="cuda", dtype=tb.TD[dtype])
    _, dW, db = jg.linear_bwd(d, A, W, needs=(False, True))
    want = sum(d[b].double().T @ A[b].double() for b in _blocks(M))
    _relative(dW, want, dtype, M)
    want = sum(d[b].double().sum(0) for b in _blocks(M))
    assert ((db.double() - want) / want).abs().max() <= 2 * tb.U * (M / 608 + 16)
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_linear_bwd_over_many_columns(jg, dtype):
    """dA over 2^20 columns of dout, in more tiles than K is split for; 16 rows
    are looked at, which differ less than a step (K entries round apart)."""
    g = torch.Generator(device="cuda").manual_seed(4)
    M, N, K = 5120, 1 << 20, 4096
    d, W = _positive(g, M, N, 1 / 64, dtype), _positive(g, N, K, 1 / 64, dtype)
    A = torch.zeros(M, K, device="cuda", dtype=tb.TD[dtype])
    dA, _, _ = jg.linear_bwd(d, A, W, bias=False, needs=(True, False))
    rows = torch.arange(M - 1, 0, -M // 16, device="cuda")
    want = sum(d[rows, b].double() @ W[b].double() for b in _blocks(N, 1 << 17))
    _relative(dA[rows], want, dtype, N, n=K)
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gated_ffn_bwd_over_many_rows(jg, dtype):
    """dWg and dWu over 2^24 rows.  dg and du are rounded to the type, at random
    over the rows, and hold fp32 errors of act and act' (32 units)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    M, D, F = 1 << 24, 64, 64
    x, dh = _positive(g, M, D, 1 / 8, dtype), _positive(g, M, F, 1 / 32, dtype)
    Wg, Wu = _positive(g, F, D, 1 / 4, dtype), _positive(g, F, D, 1 / 4, dtype)
    _, dWg, dWu, _, _ = jg.gated_ffn_bwd(dh, x, Wg, Wu, needs=(False, True, True, False, False))
    wg = wu = 0
    for b in _blocks(M):
        xb, hb = x[b].double(), dh[b].double()
        gate, up = xb @ Wg.double().T, xb @ Wu.double().T
        s = torch.sigmoid(gate)
        wg = wg + (hb * up * s * (1 + gate * (1 - s))).T @ xb
        wu = wu + (hb * gate * s).T @ xb
    # the mean of 2^24 roundings of dg, six standard deviations: 2^-12 * 6 HALF / sqrt 3
    extra = 32 * tb.U + 6 * 2.0 ** -12 * tb.HALF[dtype]
    _relative(dWg, wg, dtype, M, extra=extra)
    _relative(dWu, wu, dtype, M, extra=extra)
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", [8, 16, 20])
def test_gated_ffn_fwd_over_a_wide_row(jg, M, dtype):
    """Projections of 2^20 columns.  A relative error e of g and u is at most
    (1.3 + 1) e of h: g act'(g) / act(g) = 1 + g (1 - s) < 1.3 where g > 0."""
    g = torch.Generator(device="cuda").manual_seed(6)
    D, F = 1 << 20, 64
    x = _positive(g, M, D, 2.0 ** -9, dtype)
    Wg, Wu = _positive(g, F, D, 2.0 ** -9, dtype), _positive(g, F, D, 2.0 ** -9, dtype)
    h = jg.gated_ffn_fwd(x, Wg, Wu)
    gate, up = x.double() @ Wg.double().T, x.double() @ Wu.double().T
    want = gate * torch.sigmoid(gate) * up
    e = ((h.double() - want) / want).abs()
    assert e.max() <= tb.HALF[dtype] + 2.3 * (LONG[dtype] + (D // 512 + 32) * tb.U) + 16 * tb.U
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M", [3, 16, 20])
def test_linear_ce_fwd_over_a_wide_row(jg, M, dtype):
    """Logits of 65536 columns: lse and loss are fp32.  What a few rows' kernel
    adds is 8 warps' sums of 16 pieces; the tiles add 128 pieces."""
    g = torch.Generator(device="cuda").manual_seed(7)
    D, V = 1 << 16, 40
    x, W = _positive(g, M, D, 1 / 16, dtype), _positive(g, V, D, 1 / 64, dtype)
    lab = torch.randint(0, V, (M,), device="cuda", generator=g)
    loss, lse = jg.linear_ce_fwd(x, W, None, lab)
    z = x.double() @ W.double().T
    want = torch.logsumexp(z, 1)
    e = z.max() * (SHORT + ((24 if M <= 16 else 128) + 16) * tb.U)
    assert (lse.double() - want).abs().max() <= e, ((lse.double() - want).abs().max(), e)
    want = want - z.gather(1, lab[:, None])[:, 0]
    assert (loss.double() - want).abs().max() <= 2 * e
    jg.ops_sync()
