"""The embedding's gradient of whole numbers, whose fp32 sums are exact: runs of
one token over 7 to 3100 chunks of 16 sorted places, with the lengths next to
where they are joined by a block instead of a warp (9 or 33 chunks) and next to
1024 and 2048 chunks, which a block looks for at a time."""
import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu

MORE = [1, 7, 8, 9, 10, 31, 32, 33, 34, 511, 512, 1022, 1023, 1024, 1025, 1026, 2047, 2048, 2049, 3100]


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


def _runs():
    """Lengths of runs that go on into so many chunks after their first, with one
    place in the last of them, and with all 16; a short run between any two."""
    lengths, at = [], 0
    for k, more in enumerate(MORE):
        for end in (1, 16):
            for n in (1 + (5 * k + end) % 13, None):
                if n is None:
                    n = 16 - at % 16 + 16 * (more - 1) + end
                lengths.append(n)
                at += n
    return lengths


@pytest.mark.parametrize("dim", [24, 33, 130, 1000])
@pytest.mark.parametrize("dout_dtype,table", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16")])
def test_embedding_bwd(jg, dim, dout_dtype, table):
    runs = torch.tensor(_runs(), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(dim)
    tok = torch.repeat_interleave(torch.arange(len(runs), device="cuda"), runs)
    perm = torch.randperm(len(tok), device="cuda", generator=g)
    tok = tok[perm]
    V = len(runs) + 3
    # positive on the whole, so that a chunk that is left out or counted twice shows in every column
    d = torch.randint(-3, 8, (len(tok), dim), device="cuda", generator=g, dtype=torch.int32)
    want = torch.zeros(V, dim, device="cuda", dtype=torch.int64).index_add_(0, tok, d.long())
    assert want.abs().max() < 1 << 24
    got = jg.embedding_bwd(d.to(tb.TD[dout_dtype]), tok, V, scale=0.25, out_dtype=tb.TD[table])
    assert torch.equal(got, (want.float() * 0.25).to(tb.TD[table]))
    jg.ops_sync()


@pytest.mark.parametrize("n,dim,vocab", [(300000, 40, 3), (131073, 24, 1), (200000, 8, 40000), (70001, 4, 100)])
def test_embedding_bwd_of_few_tokens(jg, n, dim, vocab):
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    t[: n // 2] = vocab - 1
    t[torch.rand(n, device="cuda", generator=g) < 0.05] = -100
    d = torch.randint(-3, 8, (n, dim), device="cuda", generator=g, dtype=torch.int32)
    some = t >= 0
    want = torch.zeros(vocab, dim, device="cuda", dtype=torch.int64).index_add_(0, t[some], d[some].long())
    assert want.abs().max() < 1 << 24
    assert torch.equal(jg.embedding_bwd(d.float(), t, vocab), want.float())
    jg.ops_sync()
