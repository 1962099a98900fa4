"""Gates far on the negative side, where act = g Phi(g) and its slope Phi(g) + g
phi(g) are small but not zero: within bounds relative to their own size.

u = 2^-24.  Phi(g) and phi(g) come from 2^(-g^2 log2(e) / 2): the exponent's three
roundings cost 3u g^2 / 2 <= 2u g^2 of the result, the exponential 4u; what it
is multiplied by has an approximate reciprocal (2u), a fit (0.4u) and three
roundings: Phi is within (2 g^2 + 12) u of itself, phi within (1.5 g^2 + 8) u."""
import numpy as np
import pytest
import torch
from scipy.special import erfc

import training_bounds as tb

pytestmark = pytest.mark.gpu

UP = 1024.0   # the up projection: keeps fp16's h a normal number


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [9, 200])
def test_gelu_of_negative_gates(jg, rows, dtype):
    # x = (gate, 1), Wg = (1, 0), Wu = (0, UP): the projections are exact
    x = torch.zeros(rows, 8)
    x[:, 0] = torch.linspace(-8.0, -0.5, rows)
    x[:, 1] = 1.0
    x = x.to(tb.TD[dtype]).cuda()
    Wg, Wu = torch.zeros(2, 1, 8, device="cuda", dtype=tb.TD[dtype])
    Wg[0, 0], Wu[0, 1] = 1.0, UP
    g = x[:, 0].double().cpu().numpy()
    cdf, pdf = 0.5 * erfc(-g / np.sqrt(2.0)), np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)
    ecdf = cdf * ((g * g + 2) * 2 + 8) * tb.U
    h = jg.gated_ffn_fwd(x, Wg, Wu, act="gelu")[:, 0].double().cpu().numpy()
    ref = g * cdf * UP
    tb.check(h, ref, tb.rounded(ref, np.abs(g) * UP * ecdf + 4 * tb.U * np.abs(ref), dtype), "h")
    dh = torch.ones(rows, 1, device="cuda", dtype=tb.TD[dtype])
    dx = jg.gated_ffn_bwd(dh, x, Wg, Wu, act="gelu")[0].double().cpu().numpy()
    # dg = UP act'(g) and du = act(g), rounded to a 16-bit type, then dx = (dg, du UP), rounded
    slope = cdf + g * pdf
    eslope = ecdf + np.abs(g) * pdf * (1.5 * g * g + 8) * tb.U + 2 * tb.U * np.abs(slope)
    for what, got, ref, err, factor in (("dx of the gate", dx[:, 0], UP * slope, UP * eslope, 1.0),
                                        ("dx of the up", dx[:, 1], g * cdf, np.abs(g) * ecdf + 4 * tb.U * np.abs(g * cdf), UP)):
        bound = err if dtype == "f32" else tb.rounded(ref, err, dtype)
        ref, bound = ref * factor, bound * factor
        tb.check(got, ref, tb.rounded(ref, bound + 16 * tb.U * np.abs(ref), dtype), what)
    jg.ops_sync()
