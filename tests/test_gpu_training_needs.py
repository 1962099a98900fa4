"""Gradients asked for one at a time, or some of them, are those of the call
that asks for all of them, bit for bit: outputs written by the products (widths
of whole 16 bytes, many tiles), through slabs of a split K (few tiles) and
through slabs for their width (D no multiple of 8)."""
import itertools

import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


def _randn(g, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(tb.TD[dtype])


def _subsets(call, n):
    full = call((True,) * n)
    assert all(t is not None for t in full)
    for needs in itertools.product((False, True), repeat=n):
        if not any(needs):
            continue
        got = call(needs)
        for k in range(n):
            assert (got[k] is not None) == needs[k], needs
            if needs[k]:
                assert torch.equal(got[k], full[k]), (needs, k, (got[k].double() - full[k].double()).abs().max())


# rows, width, outputs: few tiles and a split K; widths of no whole 16 bytes; many tiles (direct); a wide K of z, in several pieces
SHAPES = [(300, 128, 200), (300, 130, 203), (2600, 72, 136), (2048, 1024, 1500), (5000, 512, 6000), (700, 1101, 900)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,D,F", SHAPES)
@pytest.mark.parametrize("act,bias", [("silu", True), ("gelu", False)])
def test_gated_ffn_bwd(jg, M, D, F, dtype, act, bias):
    g = torch.Generator(device="cuda").manual_seed(M + D + F)
    x, dh = _randn(g, M, D, dtype=dtype), _randn(g, M, F, dtype=dtype)
    Wg, Wu = (_randn(g, F, D, dtype=dtype, scale=D ** -0.5) for _ in range(2))
    bg, bu = (_randn(g, F) for _ in range(2)) if bias else (None, None)
    _subsets(lambda needs: jg.gated_ffn_bwd(dh, x, Wg, Wu, bg, bu, act=act, needs=needs), 5)
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,D,V", SHAPES)
@pytest.mark.parametrize("smooth", [0.0, 0.1])
def test_linear_ce_bwd(jg, M, D, V, dtype, smooth):
    g = torch.Generator(device="cuda").manual_seed(M + D + V)
    x, W, b = _randn(g, M, D, dtype=dtype), _randn(g, V, D, dtype=dtype, scale=2 * D ** -0.5), _randn(g, V)
    lab = torch.randint(0, V, (M,), device="cuda", generator=g)
    _, lse = jg.linear_ce_fwd(x, W, b, lab, smoothing=smooth)
    _subsets(lambda needs: jg.linear_ce_bwd(1.0 / M, x, W, b, lab, lse, smoothing=smooth, needs=needs), 3)
    jg.ops_sync()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_linear_bwd(jg, M, K, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    A, W, d = _randn(g, M, K, dtype=dtype), _randn(g, N, K, dtype=dtype), _randn(g, M, N, dtype=dtype)
    _subsets(lambda needs: jg.linear_bwd(d, A, W, bias=needs[2], needs=needs[:2]), 3)
    jg.ops_sync()


@pytest.mark.parametrize("dim", [96, 129, 1024, 9000])
def test_layernorm_bwd(jg, dim):
    g = torch.Generator(device="cuda").manual_seed(dim)
    for rows in (1, 40, 700):
        x, dy, w = _randn(g, rows, dim), _randn(g, rows, dim), _randn(g, dim)
        mean, rstd = x.mean(1), 1 / x.std(1)
        _subsets(lambda needs: jg.layernorm_bwd(dy, x, w, mean, rstd, needs=needs)[1:], 2)
        dx = jg.layernorm_bwd(dy, x, w, mean, rstd)[0]
        assert torch.equal(jg.layernorm_bwd(dy, x, w, mean, rstd, needs=(False, False))[0], dx)
