"""The distillation's loss where the logits have a large part in common, or the
student is close to the teacher: as a function of the z and lse that the call
returns it has the accuracy of the log-probabilities z / tau - lse, not of lse."""
import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V,K", [(1, 14, 14), (9, 300, 40), (300, 300, 300), (300, 4, 4), (40, 1000, 1000)])
@pytest.mark.parametrize("offset", [0.0, 100.0, -3000.0])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_loss_of_z_and_lse(jg, M, V, K, offset, tau, dtype):
    D = 64
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(M, D, device="cuda", generator=g).to(tb.TD[dtype])
    W = (torch.randn(V, D, device="cuda", generator=g) / 8).to(tb.TD[dtype])
    b = torch.full((V,), offset, device="cuda")
    ids = torch.rand(M, V, device="cuda", generator=g).topk(K)[1]
    # the teacher is the student but for some noise
    top = (x.float() @ W.float().T).gather(1, ids) + 0.1 * torch.randn(M, K, device="cuda", generator=g)
    loss, lse, z = jg.linear_distill_fwd(x, W, b, top, ids, temperature=tau)
    p = torch.softmax(top.double() / tau, 1)
    lq = z.double() / tau - lse.double()[:, None]
    want = tau * tau * (p * (p.log() - lq)).sum(1)
    # z / tau is rounded once (exactly halved for 2); the rest is of the size of log p and log q: a probability (10 + 8) 4u +
    # 2u (K / 32 + 16), its logarithm as much, differences and products 8u, the sum 2u (K / 32 + 16)
    size = (p * (p.log().abs() + lq.abs() + 1)).sum(1)
    tol = tau * tau * size * tb.U * (2 * 72 + 6 * (K / 32 + 16) + 8)
    assert ((loss.double() - want).abs() <= tol).all(), ((loss.double() - want).abs() / tol).max()
    jg.ops_sync()
