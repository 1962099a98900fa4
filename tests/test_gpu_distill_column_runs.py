"""The distillation's forward pass where a work unit goes over several column
tiles (2, 4 and 16 of 256 columns): the entries' logits, lse and loss of every
row, with more entries in one half of a run of tiles than are held at once (32)
and entries on the borders of halves, tiles and runs."""
import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


def _ids(M, V, K, run, g):
    """By row in turn: many of one run's left half, many of a right half, borders, the last run, anywhere."""
    def draw(n, *shape):
        return torch.randint(0, n, shape, device="cuda", generator=g)
    cols = run * 256
    r = draw(max(1, V // cols), M, 1)
    near = r * cols + draw(run, M, K) * 256 + draw(128, M, K)
    border = torch.tensor([0, 127, 128, 255], device="cuda")[draw(4, M, K)] + draw(run, M, K) * 256 + \
        draw(-(-V // cols), M, K) * cols
    edge = draw(-(-V // cols), M, K) * cols - draw(2, M, K)           # the first column of a run and the one before it
    last = V - 1 - draw(min(V, 700), M, K)
    kind = torch.arange(M, device="cuda")[:, None] % 6
    ids = draw(V, M, K)
    for k, v in enumerate((near, near + 128, border, edge, last)):
        ids = torch.where(kind == k, v, ids)
    ids = ids.clamp(0, V - 1)
    ids[torch.rand(M, K, device="cuda", generator=g) < 0.05] = -100
    ids[11] = -100
    ids[0, :] = torch.arange(K, device="cuda") + 2       # neighbours of one tile
    ids[1, :] = V - 1                                     # one class
    return ids


@pytest.mark.parametrize("dtype,M,D,V,K,run", [("bf16", 1999, 64, 390001, 80, 16), ("f16", 1999, 72, 390001, 40, 16),
                                               ("bf16", 2049, 600, 345800, 1024, 16), ("f16", 20000, 64, 9000, 80, 4),
                                               ("f32", 12001, 30, 9001, 100, 2), ("f32", 1800, 64, 390001, 70, 16)])
@pytest.mark.parametrize("bias", [True, False])
def test_linear_distill_fwd(jg, dtype, M, D, V, K, run, bias):
    tiles = -(-M // 256) * -(-V // 256)
    assert min(16, tiles // (76 * 8)) == run
    g = torch.Generator(device="cuda").manual_seed(V + K)
    x = torch.randn(M, D, device="cuda", generator=g).to(tb.TD[dtype])
    W = (torch.randn(V, D, device="cuda", generator=g) / D ** 0.5).to(tb.TD[dtype])
    b = torch.randn(V, device="cuda", generator=g) if bias else None
    top = torch.randn(M, K, device="cuda", generator=g) * 2
    ids = _ids(M, V, K, run, g)
    tau = 2.0
    loss, lse, z = jg.linear_distill_fwd(x, W, b, top, ids, temperature=tau)
    keep = ids != -100
    safe = ids.clamp(min=0)
    Wd = W.double()
    for i in range(0, M, 256):
        s = slice(i, i + 256)
        xd = x[s].double()
        full = xd @ Wd.T + (b.double() if bias else 0.0)
        size = xd.abs() @ Wd.abs().T
        # 2u (D + 16) of the terms' sizes, and 2u of the bias' addition (training_bounds.py)
        dz = 2 * tb.U * ((D + 16) * size + (b.double().abs() if bias else 0.0) + full.abs())
        ez = dz.gather(1, safe[s])
        rz = full.gather(1, safe[s]) * keep[s]
        assert ((z[s].double() - rz).abs() <= ez * keep[s]).all()
        rl = torch.logsumexp(full / tau, 1)
        q = torch.softmax(full / tau, 1)
        # as decoder_bounds.py: each term's error, its exponential's, up to 4096 additions and the joins; the logarithm
        spread = (full / tau - rl[:, None]).abs() + 2 * torch.log(torch.tensor(V + 1.0)).item()
        el = (q * (dz / tau + 2 * tb.U * (spread + 8))).sum(1) + 2 * tb.U * 4112
        el = el + 4 * tb.U * (rl.abs() + full.abs().max(1).values / tau + 1)
        assert ((lse[s].double() - rl).abs() <= el).all()
        t = torch.where(keep[s], top[s].double() / tau, torch.full_like(rz, -float("inf")))
        some = keep[s].any(1)
        p = torch.where(some[:, None], torch.softmax(t, 1), torch.zeros_like(t))
        lp = torch.where(p > 0, p.log(), torch.zeros_like(p))
        r = tau * tau * (p * (lp - (rz / tau - rl[:, None]))).sum(1)
        # probabilities: exp of differences of up to 10, a sum of K by 32 lanes, a division
        ep = (10 + 8) * 4 * tb.U + 2 * tb.U * (K / 32 + 16)
        mag = lp.abs() + rz.abs() / tau
        e = (p * (ep * (mag + rl.abs()[:, None] + 1) + ez / tau + 4 * tb.U * (mag + 8))).sum(1)
        e = e + 2 * tb.U * (K / 32 + 16) * (p * mag).sum(1) + el + 8 * tb.U * rl.abs()
        assert ((loss[s].double() - r).abs() <= (tau * tau * e + 4 * tb.U * r.abs()) * some).all()
    jg.ops_sync()
