"""Logits whose sums are exact (one-hot rows, small whole numbers).  What the
tensor core's truncation takes off a dense sum on average is given back to every
16-bit logit, so that these come out up to 0.138 n + 0.27 steps of 2^-23 of
themselves too large, n the steps of 16 products of a piece: at most 32 forward.
fp32 logits, and those of few rows, are not touched."""
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
@pytest.mark.parametrize("M,D", [(16, 512), (40, 16), (40, 512), (300, 2048)])
@pytest.mark.parametrize("rows", ["one-hot", "whole numbers"])
def test_linear_distill_z(jg, M, D, rows, dtype):
    V, K = 500, 60
    g = torch.Generator(device="cuda").manual_seed(D)
    if rows == "one-hot":
        x = torch.zeros(M, D, device="cuda")
        x[torch.arange(M, device="cuda"), torch.randint(0, D, (M,), device="cuda", generator=g)] = 1.0
        W = torch.randn(V, D, device="cuda", generator=g)
    else:
        x = torch.randint(0, 9, (M, D), device="cuda", generator=g).float()
        W = torch.randint(-3, 9, (V, D), device="cuda", generator=g).float()
    x, W = x.to(tb.TD[dtype]), W.to(tb.TD[dtype])
    ids = torch.rand(M, V, device="cuda", generator=g).topk(K)[1]
    top = torch.randn(M, K, device="cuda", generator=g)
    z = jg.linear_distill_fwd(x, W, None, top, ids, temperature=4.0)[2]
    want = (x.double() @ W.double().T).gather(1, ids)
    # one-hot fp32: W's three bf16 terms add up to it exactly
    steps = min(32, -(-D // 16))
    c = 0.0 if dtype == "f32" or M <= 16 else \
        {"bf16": 0.103 * steps + 0.07, "f16": 0.138 * steps + 0.27}[dtype] * 2.0 ** -23 + tb.U
    assert ((z.double() - want).abs() <= c * want.abs()).all()
    jg.ops_sync()
