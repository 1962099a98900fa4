"""The decoder step from a clip that the documentation shows, run as it stands
there after a small encoder, against torch's autograd in float64."""
import os
import re

import pytest
import torch

import synth
import test_gpu_decoder as base
import training_bounds as tb

pytestmark = pytest.mark.gpu

PAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
OUT = -100
jg = base.jg


@pytest.mark.parametrize("dtype,tol", [("f32", 2e-5), ("bf16", 4e-2)])
def test_step_from_a_clip(jg, dtype, tol):
    with open(PAGE) as f:
        code = re.search(r"To decode from a clip.*?```python\n(.*?)```", f.read(), re.S).group(1)
    # 135 tokens of 256 columns a clip
    cfg = synth.CONFIGS["vitl16-16f256"].with_(embed_dim=256, n_head=8, ffn_dim=512, n_layer=2, n_frames=6, height=80,
                                               width=144, batch=3)
    encoder = jg.Encoder(cfg, synth.encoder_weights(cfg))
    clip = torch.from_numpy(synth.clip_u8(cfg)).cuda()
    p, tokens, top, ids, lengths, n = base._decoder_case(dtype, B=3, T=150, D=256, C=128)
    scope = dict(p, jg=jg, torch=torch, encoder=encoder, clip=clip, tokens=tokens, lengths=lengths, top=top, ids=ids, n=n)
    exec(code, scope)
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    B, T = tokens.shape
    seen = encoder.encode(clip)["out"].double()
    encoder.sync()
    N, D = seen.shape[1:]
    assert (N, D) == (135, 256) and seen.std() > 0.1
    live = (tokens != OUT)[..., None]
    text = q["E"][tokens.clamp(min=0)] * 4.0 * live
    ln = torch.nn.functional.layer_norm
    gv = ln(torch.cat((seen, text), 1), (D,), q["w1"], q["b1"], 1e-6) @ q["Wgv"].T + q["bgv"]
    C = gv.shape[-1] // 2
    f, v, s, hs = torch.sigmoid(gv[..., :C]), gv[..., C:], torch.zeros(B, C, device="cuda", dtype=torch.float64), []
    for t in range(N + T):
        new = f[:, t] * s + (1 - f[:, t]) * v[:, t]
        s = new if t < N else torch.where(live[:, t - N], new, s)
        if t >= N:
            hs.append(s * live[:, t - N])
    x2 = text + torch.stack(hs, 1) @ q["Wo"].T + q["bo"]
    z = (ln(x2, (D,), q["w2"], q["b2"], 1e-6) @ q["Wc"].T + q["bc"]).view(B * T, -1) / 2.0
    keep = (ids != OUT).any(1)
    pt = torch.softmax(top.double() / 2.0, 1)
    kl = (pt * (torch.log(pt) - torch.log_softmax(z, 1).gather(1, ids.clamp(min=0)))).sum(1) * 4.0 * keep
    (kl.sum() / n).backward()
    # as the step without a clip: about ten roundings of half a step from the loss to the embedding
    assert (scope["loss"].double() - kl).abs().max() <= tol * kl.abs().max()
    for k in p:
        assert (scope["d" + k].double() - q[k].grad).norm() <= tol * q[k].grad.norm(), k
    # serving: the clip's rows first, then a token at a time (the recurrence alone; states of size 1, grouped otherwise)
    g = scope["gv"]
    state = jg.gated_scan_fwd(g[:, :N].contiguous(), states=False)[1]
    for t in range(N, N + 20):
        h, _, _ = jg.gated_scan_fwd(g[:, t:t + 1].contiguous(), state, states=False, last=state)
        ref = scope["h"][:, t].double()
        assert ((h[:, 0].double() - ref).abs() <= 2 * (64 * tb.U * 5 + tb.HALF[dtype] * 5)).all()
    jg.ops_sync()
    encoder.close()
