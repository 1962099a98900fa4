"""Float64 CPU restatement of the training operators (numpy, no blocking).

Layer norm, gated feed-forward, softmax cross entropy of a linear classifier
and the linear layer, with their gradients.  Shares no code with the GPU path.
"""
import numpy as np
from scipy.special import erf


def _f64(*arrays):
    return [None if a is None else np.asarray(a, np.float64) for a in arrays]


# ----------------------------------------------------------------------------- layer norm
def layer_norm_stats(x, eps):
    x, = _f64(x)
    mean = x.mean(-1)
    var = ((x - mean[..., None]) ** 2).mean(-1)
    return mean, 1.0 / np.sqrt(var + eps)


def layer_norm_bwd(dy, x, w, mean, rstd, residual=None):
    """(dx, dw, db); mean and rstd are taken as given."""
    dy, x, w, mean, rstd, residual = _f64(dy, x, w, mean, rstd, residual)
    xh = (x - mean[:, None]) * rstd[:, None]
    c = dy * w
    dx = rstd[:, None] * (c - c.mean(1, keepdims=True) - xh * (c * xh).mean(1, keepdims=True))
    if residual is not None:
        dx = dx + residual
    return dx, (dy * xh).sum(0), dy.sum(0)


# ----------------------------------------------------------------------------- linear layer
def linear_bwd(dout, A, W):
    """(dA, dW, dbias) of out = A W^T + bias."""
    dout, A, W = _f64(dout, A, W)
    return dout @ W, dout.T @ A, dout.sum(0)


# ----------------------------------------------------------------------------- softmax cross entropy
def linear_ce(x, W, bias, labels, ignore_index=-100, smoothing=0.0):
    """(loss, lse, z): loss 0 for ignored rows, NaN for labels outside [0, V)."""
    x, W, bias = _f64(x, W, bias)
    z = x @ W.T + (0.0 if bias is None else bias)
    V = z.shape[1]
    with np.errstate(invalid="ignore", divide="ignore"):
        m = z.max(1, keepdims=True)
        lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
    loss = np.full(len(z), np.nan)
    for i, y in enumerate(labels):
        if y == ignore_index:
            loss[i] = 0.0
        elif 0 <= y < V:
            loss[i] = lse[i] - (1.0 - smoothing) * z[i, y]
            if smoothing > 0.0:
                loss[i] -= smoothing * z[i].mean()
    return loss, lse, z


def linear_ce_dz(z, lse, dloss, labels, ignore_index=-100, smoothing=0.0):
    """Gradient of sum(dloss * loss) by the logits."""
    V = z.shape[1]
    dz = np.exp(z - lse[:, None]) - smoothing / V
    for i, y in enumerate(labels):
        if y == ignore_index or y < 0 or y >= V:
            dz[i] = 0.0
        else:
            dz[i, y] -= 1.0 - smoothing
            dz[i] *= dloss[i]
    return dz


# ----------------------------------------------------------------------------- gated feed-forward
def gate_act(g, act):
    if act == "silu":
        return g / (1.0 + np.exp(-g))
    return 0.5 * g * (1.0 + erf(g / np.sqrt(2.0)))


def gate_act_grad(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    return 0.5 * (1.0 + erf(g / np.sqrt(2.0))) + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)


def gated_project(x, Wg, Wu, bg=None, bu=None):
    x, Wg, Wu, bg, bu = _f64(x, Wg, Wu, bg, bu)
    return x @ Wg.T + (0.0 if bg is None else bg), x @ Wu.T + (0.0 if bu is None else bu)


def gated_ffn(x, Wg, Wu, bg=None, bu=None, act="silu"):
    g, u = gated_project(x, Wg, Wu, bg, bu)
    return gate_act(g, act) * u


def gated_ffn_bwd(dh, x, Wg, Wu, bg=None, bu=None, act="silu"):
    """(dx, dWg, dWu, dbg, dbu)."""
    dh, x, Wg, Wu = _f64(dh, x, Wg, Wu)
    g, u = gated_project(x, Wg, Wu, bg, bu)
    dg, du = dh * u * gate_act_grad(g, act), dh * gate_act(g, act)
    return dg @ Wg + du @ Wu, dg.T @ x, du.T @ x, dg.sum(0), du.sum(0)
