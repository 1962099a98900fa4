"""dbias where the rows' dloss lie far apart: the teacher's part of a class keeps
its relative accuracy next to a row whose gradient is 2^70 times as large and
has no part in the class."""
import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,V", [(300, 400), (5000, 300), (300, 2500), (9, 400)])
@pytest.mark.parametrize("far", [0, 30, 50, 70])
def test_linear_distill_dbias(jg, M, V, far, dtype):
    D, K, tau = 64, 6, 2.0
    g = torch.Generator(device="cuda").manual_seed(M + V)
    x = torch.randn(M, D, device="cuda", generator=g).to(tb.TD[dtype])
    W = (torch.randn(V, D, device="cuda", generator=g) / 8).to(tb.TD[dtype])
    b = torch.randn(V, device="cuda", generator=g)
    out = torch.tensor([3, 200, 255, 256, V - 1], device="cuda")
    b[out] = -float("inf")      # the student gives these nothing: their dbias is the teacher's part alone
    top = torch.randn(M, K, device="cuda", generator=g) * 2
    ids = torch.randint(0, V, (M, K), device="cuda", generator=g)
    ids[torch.rand(M, K, device="cuda", generator=g) < 0.1] = 256
    ids[:, 0] = out[torch.randint(0, len(out), (M,), device="cuda", generator=g)]
    ids[1] = torch.arange(10, 10 + K, device="cuda")
    dl = torch.randn(M, device="cuda", generator=g)
    dl[1] = 2.0 ** far
    loss, lse, z = jg.linear_distill_fwd(x, W, b, top, ids, temperature=tau)
    # rows that name a class twice have both probabilities
    p = torch.softmax(top.double() / tau, 1)
    term = (p * dl.double()[:, None] * tau).flatten()
    want = torch.zeros(V, device="cuda", dtype=torch.float64).index_add_(0, ids.flatten(), -term)
    size = torch.zeros(V, device="cuda", dtype=torch.float64).index_add_(0, ids.flatten(), term.abs())
    db = jg.linear_distill_bwd(dl, x, W, b, top, ids, lse, z, temperature=tau, needs=(False, False, True))[2]
    # a probability: exp of a difference of up to 10, a sum of 6, a division; its product with dloss tau / unit, three roundings; the
    # whole numbers' sum, twice rounded: (10 + 8) 4u + 2u 6 + 8u
    err = (db.double() - want).abs()
    assert (err[out] <= 92 * tb.U * size[out]).all(), (err[out] / size[out]).max() / tb.U
    jg.ops_sync()
