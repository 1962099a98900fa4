"""Element-wise error bounds of the training operators, from rounding alone.

u = 2^-24 is half an fp32 step.  An fp32 sum of K products, in any order and
with additions that round or truncate (at most 2u each), is within
2u (K + 16) sum |a b| of its value; 16 covers the rounding of the products
where an operand is split into shorter terms, joins of partial sums and bias
additions.  A value rounded to type T moves by at most eps(T)/2 of itself, or
half T's smallest subnormal.  exp by the hardware's exp2: (|argument| + 4) 2u
relative, from rounding the scaled argument and from the function's error of a
few u.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rounded(ref, err, dtype):
    """Bound after rounding a value within err of ref to dtype."""
    return err + HALF[dtype] * (np.abs(ref) + err) + TINY[dtype]


def product(a, b, aerr=None):
    """Bound of a @ b.T computed in fp32: a [M, K], b [N, K] absolute inputs,
    a known to within aerr."""
    a, b = np.abs(a), np.abs(b)
    g = 2 * U * (a.shape[1] + 16)
    e = g * (a @ b.T)
    if aerr is not None:
        e = e + (1 + g) * (aerr @ b.T)
    return e


def check(got, ref, bound, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))   # infinities and NaN where they belong
    bad = ~same & ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = tuple(int(k) for k in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: got {got[i]!r}, expected "
                             f"{ref[i]!r} within {np.broadcast_to(bound, ref.shape)[i]:.3g}")


# ----------------------------------------------------------------------------- cross entropy
def ce_logits(x, W, bias):
    """Bound of the fp32 logits."""
    e = product(x, W)
    if bias is not None:
        z = np.abs(np.where(np.isfinite(bias), bias, 0.0))
        e = e + 2 * U * (z + np.abs(x @ W.T))
    return e


def ce_forward(x, W, bias, z, lse, loss, labels, smoothing):
    """Bounds of (loss, lse)."""
    V = z.shape[1]
    dz = ce_logits(x, W, bias)
    fin = np.where(np.isfinite(z), z, 0.0)
    p = np.exp(np.where(np.isfinite(z), z - lse[:, None], -np.inf))
    # relative error of sum exp(z - m): each term's dz and exp, V additions; then log and the final sum
    spread = np.abs(fin - lse[:, None]) + 2 * np.log(V + 1)
    rel = (p * (dz + 2 * U * (spread + 8))).sum(1) + 2 * U * (min(V, 4096) + 16) * p.sum(1)
    elise = rel + 4 * U * (np.abs(lse) + np.abs(fin).max(1) + 1)
    y = np.clip(labels, 0, V - 1)
    r = np.arange(len(z))
    el = elise + dz[r, y] + 4 * U * (np.abs(fin[r, y]) + np.abs(lse))
    if smoothing > 0:
        el = el + smoothing * (dz.mean(1) + 2 * U * (min(V, 4096) + 16) * np.abs(fin).mean(1)) + 4 * U * np.abs(fin).mean(1)
    return el, elise


def ce_dz(x, W, bias, z, lse, dloss, labels, smoothing, dtype):
    """(dz bound in fp32, dz bound after rounding to dtype)."""
    e = ce_logits(x, W, bias)
    fin = np.where(np.isfinite(z), z, 0.0)
    p = np.where(np.isfinite(z), np.exp(z - lse[:, None]), 0.0)
    arg = e + 4 * U * (np.abs(fin) + np.abs(lse)[:, None] + 4)
    dp = p * (np.expm1(arg)) + 2 * U
    dp = np.where(p == 0, 2 * U, dp)
    dl = np.abs(dloss)[:, None]
    err = dl * (dp + 6 * U * (p + 1.0 * (np.arange(z.shape[1])[None] == np.asarray(labels)[:, None]) + smoothing))
    return err


# ----------------------------------------------------------------------------- gate
def gate(g, u, eg, eu, act):
    """Bounds of act(g) and act'(g) in fp32 for a g known to within eg."""
    slope = 1.13 if act == "gelu" else 1.10      # largest |act'|
    curve = 0.8 if act == "gelu" else 0.5        # largest |act''|
    ea = slope * eg + (np.abs(g) + 8) * 4 * U * np.minimum(np.abs(g) + 1, 40)
    ed = curve * eg + (np.abs(g) + 8) * 8 * U
    return ea, ed
