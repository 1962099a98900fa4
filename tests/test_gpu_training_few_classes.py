"""dbias of few classes and many rows.  Its rows' entries p - [v = label] cancel
over the rows, an error of z of one sign (the tensor core's truncation) does
not: with 128 rows a class and more, z is taken out of the accumulator every 128
products, 8 steps, and from 32 rows on every 256, 16 steps.  n < 40 steps of
products of one sign cost z at most (n + 2) 2^-23 of itself (measured)."""
import numpy as np
import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu



@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("signs", ["positive", "halfnormal"])
@pytest.mark.parametrize("M,D,V,steps", [(100000, 768, 12, 8), (30000, 768, 12, 8), (3000, 768, 12, 8), (1789, 448, 12, 8),
                                         (100000, 1536, 300, 8), (100000, 1024, 1000, 16)])
def test_linear_ce_dbias(jg, M, D, V, steps, signs, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + V)
    # same-signed products: z of about 13 (D 768) and 27, not far from alike for all classes
    def draw(*shape):
        return 0.5 + 0.5 * torch.rand(*shape, device="cuda", generator=g) if signs == "positive" else \
            torch.randn(*shape, device="cuda", generator=g).abs()
    x = draw(M, D).to(tb.TD[dtype])
    W = (draw(V, D) / 32).to(tb.TD[dtype])
    lab = torch.randint(0, V, (M,), device="cuda", generator=g)
    z = x.double() @ W.double().T
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    want = p.sum(0) - torch.bincount(lab, minlength=V)
    top = z.max()
    # of one sign: z's truncation, and exp2's error of 2 units; at random over the rows, six standard deviations of
    # half steps: the rounding of lse and of the scaled z and lse, and of z's sums (D / 128 of them); 40 additions
    # of each strip and join
    one = p.sum(0) * (top * (steps + 2) * 2 * tb.U + 4 * tb.U)
    rnd = 6 * p.square().sum(0).sqrt() * top * 2 * tb.U * np.sqrt(3 + D / 128)
    add = 2 * tb.U * 40 * (want.abs() + 6 * np.sqrt(M / V))
    for l in (lse.float(), jg.linear_ce_fwd(x, W, None, lab)[1]):
        _, _, db = jg.linear_ce_bwd(1.0, x, W, None, lab, l)
        e = (db.double() - want).abs()
        assert (e <= one + rnd + add).all(), (e.max(), one.max(), rnd.max(), add.max())
    jg.ops_sync()
