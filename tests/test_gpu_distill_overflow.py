"""A logit whose sum of products overflows to -infinity gives its class no
probability, in every type and for few rows and many, as in the cross entropy."""
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
@pytest.mark.parametrize("M", [16, 17, 300])
@pytest.mark.parametrize("bias", [True, False])
def test_a_class_whose_logit_overflows(jg, M, bias, dtype):
    D, V, K, out = 64, 400, 5, 270
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, D, device="cuda", generator=g)
    W = torch.randn(V, D, device="cuda", generator=g) / 8
    # powers of two: one term of one sign, nothing to cancel; every other class has a 0 there
    W[:, 0] = 0
    x[:, 0], W[out, 0] = 2.0 ** 100, -2.0 ** 100
    x, W = x.to(tb.TD[dtype]), W.to(tb.TD[dtype])
    b = torch.randn(V, device="cuda", generator=g) if bias else None
    top = torch.randn(M, K, device="cuda", generator=g)
    ids = torch.randint(0, out, (M, K), device="cuda", generator=g)
    loss, lse, z = jg.linear_distill_fwd(x, W, b, top, ids, temperature=2.0)
    full = x.double() @ W.double().T + (b.double() if bias else 0.0)
    full[:, out] = -float("inf")
    # 63 products and 16 of joins of logits of size 10, sums of 400 terms: 2u (80 + 400) 10 at most
    tol = 2 * tb.U * 480 * 10
    assert (lse.double() - torch.logsumexp(full / 2, 1)).abs().max() <= tol
    assert (z.double() - full.gather(1, ids)).abs().max() <= tol
    p = torch.softmax(top.double() / 2, 1)
    logq = torch.log_softmax(full / 2, 1).gather(1, ids)
    assert (loss.double() - 4 * (p * (p.log() - logq)).sum(1)).abs().max() <= 4 * 4 * tol
    dx, dW, db = jg.linear_distill_bwd(1.0, x, W, b, top, ids, lse, z, temperature=2.0)
    dz = torch.softmax(full / 2, 1).scatter_add_(1, ids, -p) * 2
    assert db[out] == 0 and (db.double() - dz.sum(0)).abs().max() <= 2 * M * tol
    # dW of column 0, whose x is 2^100, is not compared; dx's other columns are those without the class
    h = tb.HALF[dtype]
    rx, rw = dz @ W.double(), dz.T @ x.double()
    assert not dW[out].any() and torch.isfinite(dx).all()
    assert (dx.double() - rx)[:, 1:].norm() <= (2 * h + 1e-4) * rx[:, 1:].norm()
    assert (dW.double() - rw)[:, 1:].norm() <= (2 * h + 1e-4) * rw[:, 1:].norm()
    # a teacher that names the class: an infinite loss, and the gradient of its probability
    ids[3, 0] = out
    loss, lse2, z = jg.linear_distill_fwd(x, W, b, top, ids, temperature=2.0)
    assert loss[3] == float("inf") and z[3, 0] == -float("inf") and torch.equal(lse, lse2)
    assert torch.isfinite(torch.cat([loss[:3], loss[4:]])).all()
    db = jg.linear_distill_bwd(1.0, x, W, b, top, ids, lse, z, temperature=2.0, needs=(False, False, True))[2]
    assert abs(float(db[out]) + 2 * float(p[3, 0])) <= 2 * 92 * tb.U   # of a probability: (10 + 8) 4u + 2u 5 and a few roundings
    jg.ops_sync()
