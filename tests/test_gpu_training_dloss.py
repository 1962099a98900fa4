"""A dloss that is not finite stays in its row's dx."""
import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M", [150, 20000])   # dz's unit found by the product, and by its own kernel
@pytest.mark.parametrize("scale", [1e-6, 30.0])
def test_row_of_infinite_dloss(jg, M, dtype, scale):
    g = torch.Generator(device="cuda").manual_seed(M)
    D, V, row = 64, 300, 77
    x = torch.randn(M, D, device="cuda", generator=g).to(tb.TD[dtype])
    W = (torch.randn(V, D, device="cuda", generator=g) / 4).to(tb.TD[dtype])
    lab = torch.randint(0, V, (M,), device="cuda", generator=g)
    dl = torch.randn(M, device="cuda", generator=g) * scale
    _, lse = jg.linear_ce_fwd(x, W, None, lab)
    dl[row] = 0.0
    want = jg.linear_ce_bwd(dl, x, W, None, lab, lse)[0]
    assert torch.isfinite(want).all()
    others = torch.arange(M, device="cuda") != row
    for v in (float("inf"), float("-inf"), float("nan")):
        dl[row] = v
        got = jg.linear_ce_bwd(dl, x, W, None, lab, lse)[0]
        assert torch.equal(got[others], want[others]), v
        assert not torch.isfinite(got[row]).any()
    jg.ops_sync()
