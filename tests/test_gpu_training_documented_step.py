"""The training step that the documentation shows, run as it stands there, at
widths that it names as allowed; and what it says of autograd."""
import os
import re

import numpy as np
import pytest
import torch

import test_gpu_training as base

pytestmark = pytest.mark.gpu

PAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
jg = base.jg


@pytest.mark.parametrize("dim,hidden", [(1024, 2752), (384, 1024)])
def test_training_step(jg, dim, hidden):
    with open(PAGE) as f:
        code = re.search(r"A training step of one gated MLP block.*?```python\n(.*?)```", f.read(), re.S).group(1)
    rng = np.random.default_rng(dim)
    rows, classes = 300, 174
    p, _ = base._block_params(rng, dim, hidden, classes, "bf16")
    x = torch.randn(rows, dim, device="cuda")
    labels = torch.randint(0, classes, (rows,), device="cuda")
    scope = dict(p, jg=jg, torch=torch, x=x, labels=labels, n=rows)
    exec(code, scope)
    loss, grads = base._block(jg, p, x, labels, rows)
    assert torch.equal(scope["loss"], loss)
    for name, g in grads.items():
        assert torch.equal(scope["d" + name], g), name
    jg.ops_sync()


def test_results_carry_no_graph(jg):
    x = torch.randn(40, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    y, _, _ = jg.layernorm_fwd(x, w, torch.zeros(64, device="cuda"), 1e-6)
    assert not y.requires_grad
    for shift in (0, 1):   # also where an operand is copied to 16 bytes
        W = torch.randn(200 * 64 + shift, device="cuda", requires_grad=True)[shift:].view(200, 64)
        loss, lse = jg.linear_ce_fwd(x, W, None, torch.zeros(40, dtype=torch.int64, device="cuda"))
        grads = jg.linear_ce_bwd(1.0, x, W, None, torch.zeros(40, dtype=torch.int64, device="cuda"), lse)
        assert not any(t.requires_grad for t in (loss, lse) + grads), shift
        h = jg.gated_ffn_fwd(x, W, W)
        grads = jg.gated_ffn_bwd(torch.ones_like(h), x, W, W)
        assert not any(t.requires_grad for t in (h,) + grads), shift
        assert not any(t.requires_grad for t in jg.linear_bwd(h, x, W)), shift
