"""The gated recurrence over many pieces, element by element within the bounds of
decoder_bounds.py, which are made here step by step on the device: long
sequences, and tensors whose offsets pass 2^31 elements."""
import pytest
import torch

import training_bounds as tb

pytestmark = pytest.mark.gpu

U, LEVELS = tb.U, 16


@pytest.fixture(scope="module")
def jg():
    import video_vit_encoder_gb300 as m
    m.load()
    return m


def _near(got, ref, err, half, tiny):
    return ((got.double() - ref).abs() <= err + half * (ref.abs() + err) + tiny).all()


# batch, steps, width, type, mean gate, lengths
CASES = [(1, 9999, 33, "f16", 3.0, False), (2, 5000, 70, "bf16", 3.0, True), (3, 4609, 777, "f32", 2.0, False),
         (3, 4609, 777, "bf16", 2.0, True), (8, 2048, 1024, "bf16", 2.0, True), (1, 6000, 256, "bf16", 6.0, False),
         (40, 300, 778, "f16", 2.0, True), (2, 600, 1 << 20, "bf16", 2.0, False), (2, 700, (1 << 20) - 3, "f16", 2.0, True)]


@pytest.mark.parametrize("B,T,C,dtype,mean,ragged", CASES)
def test_gated_scan(jg, B, T, C, dtype, mean, ragged):
    g = torch.Generator(device="cuda").manual_seed(T + C)
    dt, half, tiny = tb.TD[dtype], tb.HALF[dtype], tb.TINY[dtype]
    gv = torch.randn(B, T, 2 * C, device="cuda", generator=g, dtype=dt)
    gv[..., :C].mul_(1.5).add_(mean)
    dh = torch.randn(B, T, C, device="cuda", generator=g, dtype=dt)
    h0, dl = torch.randn(B, C, device="cuda", generator=g), torch.randn(B, C, device="cuda", generator=g)
    n = torch.full((B,), T, device="cuda", dtype=torch.int32)
    if ragged:
        n[:-1] = torch.randint(0, T + 1, (B - 1,), device="cuda", generator=g, dtype=torch.int32)
    lengths = n if ragged else None
    h, last, states = jg.gated_scan_fwd(gv, h0, lengths=lengths)

    def step(t):
        x = gv[:, t, :C].double()
        live = (t < n)[:, None]
        return torch.sigmoid(x), torch.sigmoid(-x), (1.2 * x.abs() + 8) * 2 * U, gv[:, t, C:].double(), live
    # the state before each step, and what is known of it, for the backward pass
    before = torch.empty(B, T, C, device="cuda", dtype=torch.float64 if C < 1 << 19 else torch.float32)
    known = torch.empty(B, T, C, device="cuda")
    x, size, e = h0.double(), h0.double().abs(), torch.zeros(B, C, device="cuda", dtype=torch.float64)
    for t in range(T):
        f, k, eta, v, live = step(t)
        if t % 128 == 0:
            assert _near(states[:, t // 128], x, e + LEVELS * 4 * U * size, 0.0, 0.0), t
        before[:, t], known[:, t] = x, e + LEVELS * 4 * U * size
        e = torch.where(live, f * (e + (eta + 4 * U) * size) + k * v.abs() * (eta + 4 * U), e)
        size = torch.where(live, f * size + k * v.abs(), size)
        x = torch.where(live, f * x + k * v, x)
        ok = (h[:, t].double() - x).abs() <= e + LEVELS * 4 * U * size + half * (x.abs() + e + LEVELS * 4 * U * size) + tiny
        assert torch.where(live, ok, h[:, t] == 0).all(), t
    assert _near(last, x, e + LEVELS * 4 * U * size, 0.0, 0.0)
    dgv, dh0 = jg.gated_scan_bwd(dh, gv, states, lengths=lengths, dlast=dl)
    # before is kept in fp32 where it would not fit otherwise: u of it more
    more = 0.0 if before.dtype == torch.float64 else U
    l, size, e = dl.double(), dl.double().abs(), torch.zeros(B, C, device="cuda", dtype=torch.float64)
    for t in range(T - 1, -1, -1):
        f, k, eta, v, live = step(t)
        here, hsize = l + dh[:, t].double(), size + dh[:, t].double().abs()
        el = e + LEVELS * 4 * U * hsize + 2 * U * here.abs()
        dv, ev = here * k, el * k + here.abs() * k * (eta + 4 * U)
        b = before[:, t].double()
        diff = b - v
        dg = dv * f * diff
        # the kept states are within `known` of the exact ones, and the states made from them as much again
        eg = f * (el * k * diff.abs() + dv.abs() * (2 * known[:, t] + more * b.abs() + 2 * U * (b.abs() + v.abs())) +
                  dv.abs() * diff.abs() * (2 * eta + 8 * U))
        for got, ref, err in ((dgv[:, t, :C], dg, eg), (dgv[:, t, C:], dv, ev)):
            ok = (got.double() - ref).abs() <= err + half * (ref.abs() + err) + tiny
            assert torch.where(live, ok, got == 0).all(), t
        l = torch.where(live, f * here, l)
        e = torch.where(live, f * (e + (eta + 4 * U) * hsize), e)
        size = torch.where(live, f * hsize, size)
    assert _near(dh0, l, e + LEVELS * 4 * U * size, 0.0, 0.0)
    jg.ops_sync()
