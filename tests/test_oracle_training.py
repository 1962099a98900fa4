"""The training oracle: gradients against central differences of its forward
functions and against torch's float64 autograd, and the corner cases of the
cross entropy (ignored and bad labels, masked classes, smoothing)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import training as ot


def _diff(f, a, eps=1e-6):
    """Central differences of the scalar f() by every element of a (in place)."""
    g = np.zeros_like(a)
    it = np.nditer(a, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = a[i]
        a[i] = keep + eps
        hi = f()
        a[i] = keep - eps
        lo = f()
        a[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


def _close(got, ref):
    # differences at step 1e-6 of values of order 1: rounding 1e-16 / 1e-6 and a third-derivative term of 1e-12,
    # with room for the sums over a few dozen terms
    assert np.abs(got - ref).max() <= 1e-7 * max(1.0, np.abs(ref).max())


def test_layer_norm_gradients():
    rng = np.random.default_rng(0)
    x, w, b, dy, res = (rng.standard_normal(s) for s in ((4, 7), (7,), (7,), (4, 7), (4, 7)))

    def f():
        return (oracle.layer_norm(x, w, b, 1e-6) * dy).sum()
    mean, rstd = ot.layer_norm_stats(x, 1e-6)
    dx, dw, db = ot.layer_norm_bwd(dy, x, w, mean, rstd)
    for got, a in ((dx, x), (dw, w), (db, b)):
        _close(got, _diff(f, a))
    np.testing.assert_allclose(ot.layer_norm_bwd(dy, x, w, mean, rstd, res)[0], dx + res)


def test_layer_norm_one_column():
    """One column: y = b whatever x is, so dx = 0."""
    x = np.array([[3.0], [-2.0]])
    mean, rstd = ot.layer_norm_stats(x, 1e-6)
    dx, dw, db = ot.layer_norm_bwd(np.ones((2, 1)), x, np.ones(1), mean, rstd)
    assert np.all(dx == 0) and dw[0] == 0 and db[0] == 2


def test_linear_gradients():
    rng = np.random.default_rng(1)
    A, W, b, d = (rng.standard_normal(s) for s in ((5, 3), (4, 3), (4,), (5, 4)))

    def f():
        return ((A @ W.T + b) * d).sum()
    for got, a in zip(ot.linear_bwd(d, A, W), (A, W, b)):
        _close(got, _diff(f, a))


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_cross_entropy_gradients(smoothing):
    rng = np.random.default_rng(2)
    x, W, b, dl = (rng.standard_normal(s) for s in ((5, 3), (6, 3), (6,), (5,)))
    labels = np.array([2, -100, 0, 5, 2])

    def f():
        return (ot.linear_ce(x, W, b, labels, smoothing=smoothing)[0] * dl).sum()
    _, lse, z = ot.linear_ce(x, W, b, labels, smoothing=smoothing)
    dz = ot.linear_ce_dz(z, lse, dl, labels, smoothing=smoothing)
    for got, a in ((dz @ W, x), (dz.T @ x, W), (dz.sum(0), b)):
        _close(got, _diff(f, a))


@pytest.mark.parametrize("smoothing", [0.0, 0.2])
def test_cross_entropy_against_torch(smoothing):
    rng = np.random.default_rng(3)
    x, W, b = rng.standard_normal((9, 4)), rng.standard_normal((11, 4)), rng.standard_normal(11)
    labels = rng.integers(0, 11, 9)
    labels[4] = -100
    t = torch.nn.functional.cross_entropy(torch.from_numpy(x @ W.T + b), torch.from_numpy(labels),
                                          reduction="none", label_smoothing=smoothing)
    loss, lse, z = ot.linear_ce(x, W, b, labels, smoothing=smoothing)
    np.testing.assert_allclose(loss, t.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(torch.from_numpy(z), 1).numpy(), rtol=1e-12)


def test_cross_entropy_masked_class_and_bad_label():
    rng = np.random.default_rng(4)
    x, W, b = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), np.array([0, -np.inf, 0, 0, 0.0])
    loss, lse, z = ot.linear_ce(x, W, b, [0, 5, -1])
    keep = [0, 2, 3, 4]
    np.testing.assert_allclose(lse, np.log(np.exp(z[:, keep]).sum(1)))
    assert np.isfinite(loss[0]) and np.isnan(loss[1]) and np.isnan(loss[2])
    dz = ot.linear_ce_dz(z, lse, np.ones(3), [0, 5, -1])
    assert np.all(dz[:, 1] == 0) and np.all(dz[1:] == 0)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_ffn_gradients(act):
    rng = np.random.default_rng(5)
    x, Wg, Wu, bg, bu, dh = (rng.standard_normal(s) for s in ((4, 3), (5, 3), (5, 3), (5,), (5,), (4, 5)))

    def f():
        return (ot.gated_ffn(x, Wg, Wu, bg, bu, act) * dh).sum()
    for got, a in zip(ot.gated_ffn_bwd(dh, x, Wg, Wu, bg, bu, act), (x, Wg, Wu, bg, bu)):
        _close(got, _diff(f, a))
    tg = torch.nn.functional.silu if act == "silu" else torch.nn.functional.gelu
    g = np.linspace(-6, 6, 41)
    np.testing.assert_allclose(ot.gate_act(g, act), tg(torch.from_numpy(g)).numpy(), rtol=1e-12, atol=1e-15)
