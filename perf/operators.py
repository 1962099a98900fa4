"""The training operators, measured: plain forms, the library's kernels, sizes.

The operators are what training a head on the encoder's tokens needs beside
the forward passes: layer norm forward and backward, the gated feed-forward
forward and backward, the linear layer's backward, and the softmax cross
entropy of a linear classifier over a large vocabulary with its gradients.

``run`` is one pass through one of them: in elementary 32-bit torch operations
when ``own`` is false, through the package's entry points when it is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100
EPS = 1e-6


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # the first norm of a block: 8 clips x 2048 tokens of the fp32 residual stream, normalised to the
        # 16-bit input of a matrix product
        {"name": "ln_fwd_tokens", "op": "ln_fwd", "rows": 16384, "dim": 1024, "x": "f32", "y": "bf16"},
        # its backward pass: 16-bit gradient in, fp32 residual gradient added and passed on
        {"name": "ln_bwd_tokens", "op": "ln_bwd", "rows": 16384, "dim": 1024, "x": "f32", "y": "bf16", "res": True},
        # a predictor-sized odd width in one 16-bit type, four long clips of 18432 tokens
        {"name": "ln_bwd_long", "op": "ln_bwd", "rows": 73728, "dim": 777, "x": "bf16", "y": "bf16", "res": False},
        # the classifier of the attentive-pool head, one row per clip, in fp32
        {"name": "ce_fwd_head", "op": "ce_fwd", "rows": 8, "dim": 1024, "vocab": 174, "dtype": "f32", "smooth": 0.1},
        # next-token loss of a captioning head over a large vocabulary
        {"name": "ce_fwd_large", "op": "ce_fwd", "rows": 8192, "dim": 2048, "vocab": 131072, "dtype": "bf16",
         "smooth": 0.0},
        # its gradients over a vocabulary of no round size, the last batch of an epoch
        {"name": "ce_bwd_ragged", "op": "ce_bwd", "rows": 1999, "dim": 768, "vocab": 50021, "dtype": "bf16",
         "smooth": 0.0},
        # masked-token training against a codebook with smoothed labels, fp16 under a loss scale
        {"name": "ce_bwd_smooth", "op": "ce_bwd", "rows": 4096, "dim": 1024, "vocab": 32768, "dtype": "f16",
         "smooth": 0.1},
        # a gated feed-forward on 8 clips' tokens; hidden width 2/3 of 4 x 1024, rounded up to 16
        {"name": "ffn_fwd_tokens", "op": "ffn_fwd", "rows": 16384, "dim": 1024, "hidden": 2736, "dtype": "bf16",
         "act": "silu", "bias": False},
        # the same on one pooled row per clip: the weights are all the traffic
        {"name": "ffn_fwd_pooled", "op": "ffn_fwd", "rows": 8, "dim": 1024, "hidden": 4096, "dtype": "bf16",
         "act": "gelu", "bias": True},
        # its backward pass on a batch of tokens
        {"name": "ffn_bwd_tokens", "op": "ffn_bwd", "rows": 16384, "dim": 1024, "hidden": 2736, "dtype": "bf16",
         "act": "silu", "bias": True},
        # the 2.1 predictor's projection 384 -> 1664 on half of a 4608-token clip, fp16
        {"name": "linear_bwd_proj", "op": "linear_bwd", "rows": 2304, "n": 1664, "k": 384, "dtype": "f16",
         "bias": False},
        # a down projection's gradients, fp32 and a ragged batch (one clip of 14 x 14 x 8 tokens)
        {"name": "linear_bwd_f32", "op": "linear_bwd", "rows": 1568, "n": 768, "k": 2048, "dtype": "f32",
         "bias": True},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ce_fwd", "ce_bwd", "ffn_fwd", "ffn_bwd", "linear_bwd"])
    if op.startswith("ln"):
        rows, dim = _log_int(rng, 1, 73728), _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            dim = max(64, dim // 64 * 64)
        rows = max(1, min(rows, 73728 * 1024 // dim))
        x, y = rng.choice([("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
        case = {"op": op, "rows": rows, "dim": dim, "x": x, "y": y}
        if op == "ln_bwd":
            case["res"] = rng.random() < 0.5
        return case
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    # products of one pass: within the largest listed case, and less where fp32 is asked for
    cap = 4e12 if dtype != "f32" else 3e11
    if op.startswith("ce"):
        rows, dim, vocab = _log_int(rng, 1, 8192), _log_int(rng, 64, 2048, 8), _log_int(rng, 2, 131072)
        per_row = (2 if op == "ce_fwd" else 6) * dim * vocab
        return {"op": op, "rows": max(1, min(rows, int(cap / per_row))), "dim": dim, "vocab": vocab, "dtype": dtype,
                "smooth": rng.choice([0.0, 0.0, 0.1])}
    if op == "linear_bwd":
        rows, n, k = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192, 8), _log_int(rng, 64, 8192, 8)
        return {"op": op, "rows": max(1, min(rows, int(cap / (4 * n * k)))), "n": n, "k": k, "dtype": dtype,
                "bias": rng.random() < 0.7}
    rows, dim, hidden = _log_int(rng, 1, 16384), _log_int(rng, 64, 2048, 8), _log_int(rng, 64, 8192, 8)
    per_row = (4 if op == "ffn_fwd" else 12) * dim * hidden
    return {"op": op, "rows": max(1, min(rows, int(cap / per_row))), "dim": dim, "hidden": hidden, "dtype": dtype,
            "act": rng.choice(["silu", "gelu"]), "bias": rng.random() < 0.7}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))


def _randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op, rows = case["op"], case["rows"]
    st = {"op": op}
    if op.startswith("ln"):
        dim = case["dim"]
        # a residual stream: rows with their own offset and size, a few large channels
        x = _randn(g, rows, dim) * (0.5 + torch.rand(rows, 1, device="cuda", generator=g))
        x = x + _randn(g, rows, 1, scale=0.3)
        x[:, :: max(dim // 4, 1)] *= 8.0
        st["x"] = x.to(DTYPES[case["x"]])
        st["w"] = 1.0 + _randn(g, dim, scale=0.1)
        st["b"] = _randn(g, dim, scale=0.1)
        st["y_dtype"] = DTYPES[case["y"]]
        if op == "ln_bwd":
            st["dy"] = _randn(g, rows, dim, scale=0.05, dtype=DTYPES[case["y"]])
            st["res"] = _randn(g, rows, dim, scale=0.05, dtype=DTYPES[case["x"]]) if case["res"] else None
            st["mean"], st["rstd"] = _ln_stats(st["x"])
        return st
    dt = DTYPES[case["dtype"]]
    # fp16 training runs under a loss scale, so its gradients are larger
    gscale = 0.25 if case["dtype"] == "f16" else 0.01
    if op.startswith("ce"):
        dim, vocab = case["dim"], case["vocab"]
        st["x"] = _randn(g, rows, dim, dtype=dt)
        st["w"] = _randn(g, vocab, dim, scale=2.0 / math.sqrt(dim), dtype=dt)
        st["b"] = _randn(g, vocab, scale=0.5)
        labels = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
        ignored = torch.rand(rows, device="cuda", generator=g) < 0.1
        st["labels"] = torch.where(ignored, torch.full_like(labels, IGNORE), labels)
        st["smooth"] = case["smooth"]
        if op == "ce_bwd":
            # the gradient of the mean over the rows that count, under the loss scale in fp16
            n = (st["labels"] != IGNORE).sum().clamp(min=1).float()
            loss_scale = 65536.0 if case["dtype"] == "f16" else 1.0
            st["dloss"] = (loss_scale / n).expand(rows).contiguous()
            st["lse"] = torch.cat([_logsumexp(_logits(st["x"][r:r + 1024], st["w"], st["b"]))
                                   for r in range(0, rows, 1024)])
        return st
    if op == "linear_bwd":
        n, k = case["n"], case["k"]
        st["a"] = _randn(g, rows, k, dtype=dt)
        st["w"] = _randn(g, n, k, scale=1.0 / math.sqrt(k), dtype=dt)
        st["dy"] = _randn(g, rows, n, scale=gscale, dtype=dt)
        st["bias"] = case["bias"]
        return st
    dim, hidden = case["dim"], case["hidden"]
    st["x"] = _randn(g, rows, dim, dtype=dt)
    st["wg"] = _randn(g, hidden, dim, scale=1.0 / math.sqrt(dim), dtype=dt)
    st["wu"] = _randn(g, hidden, dim, scale=1.0 / math.sqrt(dim), dtype=dt)
    st["bg"] = _randn(g, hidden, scale=0.2) if case["bias"] else None
    st["bu"] = _randn(g, hidden, scale=0.2) if case["bias"] else None
    st["act"] = case["act"]
    if op == "ffn_bwd":
        st["dh"] = _randn(g, rows, hidden, scale=gscale, dtype=dt)
    return st


# ----------------------------------------------------------------------------- plain forms (32 bits)
def _ln_stats(x):
    x = x.float()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    return mean, 1.0 / torch.sqrt(var + EPS)


def _ln_fwd(st):
    x = st["x"].float()
    mean, rstd = _ln_stats(x)
    y = (x - mean[:, None]) * rstd[:, None] * st["w"] + st["b"]
    return {"y": y.to(st["y_dtype"]), "mean": mean, "rstd": rstd}


def _ln_bwd(st):
    x, dy = st["x"].float(), st["dy"].float()
    rstd = st["rstd"][:, None]
    xh = (x - st["mean"][:, None]) * rstd
    c = dy * st["w"]
    dx = rstd * (c - c.mean(1, keepdim=True) - xh * (c * xh).mean(1, keepdim=True))
    if st["res"] is not None:
        dx = dx + st["res"].float()
    return {"dx": dx.to(st["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _logits(x, w, b):
    return x.float() @ w.float().T + b


def _logsumexp(z):
    m = z.max(1).values
    return m + torch.log(torch.exp(z - m[:, None]).sum(1))


def _ce_fwd(st):
    z = _logits(st["x"], st["w"], st["b"])
    lse = _logsumexp(z)
    valid = st["labels"] != IGNORE
    y = st["labels"].clamp(min=0)
    s = st["smooth"]
    loss = lse - (1.0 - s) * z.gather(1, y[:, None])[:, 0]
    if s > 0.0:
        loss = loss - s * z.mean(1)
    return {"loss": torch.where(valid, loss, torch.zeros_like(loss)), "lse": lse}


def _ce_bwd(st):
    x, w = st["x"].float(), st["w"].float()
    dz = torch.exp(x @ w.T + st["b"] - st["lse"][:, None])
    valid = st["labels"] != IGNORE
    y = st["labels"].clamp(min=0)
    s = st["smooth"]
    if s > 0.0:
        dz = dz - s / dz.shape[1]
    r = torch.arange(dz.shape[0], device=dz.device)
    dz[r, y] -= 1.0 - s
    dz = dz * torch.where(valid, st["dloss"], torch.zeros_like(st["dloss"]))[:, None]
    dt = st["x"].dtype
    return {"dx": (dz @ w).to(dt), "dw": (dz.T @ x).to(dt), "db": dz.sum(0)}


def _act(g, name):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))


def _act_grad(g, name):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    phi = torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * phi


def _project(x, w, b):
    z = x @ w.T
    return z if b is None else z + b


def _ffn_fwd(st):
    x = st["x"].float()
    g = _project(x, st["wg"].float(), st["bg"])
    u = _project(x, st["wu"].float(), st["bu"])
    return (_act(g, st["act"]) * u).to(st["x"].dtype)


def _ffn_bwd(st):
    x, wg, wu, dh = st["x"].float(), st["wg"].float(), st["wu"].float(), st["dh"].float()
    g = _project(x, wg, st["bg"])
    u = _project(x, wu, st["bu"])
    dg = dh * u * _act_grad(g, st["act"])
    du = dh * _act(g, st["act"])
    dt = st["x"].dtype
    out = {"dx": (dg @ wg + du @ wu).to(dt), "dwg": (dg.T @ x).to(dt), "dwu": (du.T @ x).to(dt)}
    if st["bg"] is not None:
        out["dbg"], out["dbu"] = dg.sum(0), du.sum(0)
    return out


def _linear_bwd(st):
    a, w, dy = st["a"].float(), st["w"].float(), st["dy"].float()
    dt = st["a"].dtype
    out = {"da": (dy @ w).to(dt), "dw": (dy.T @ a).to(dt)}
    if st["bias"]:
        out["db"] = dy.sum(0)
    return out


PLAIN = {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "ce_fwd": _ce_fwd, "ce_bwd": _ce_bwd, "ffn_fwd": _ffn_fwd,
         "ffn_bwd": _ffn_bwd, "linear_bwd": _linear_bwd}


# ----------------------------------------------------------------------------- the library's kernels
def _own(st):
    import video_vit_encoder_gb300 as jg

    op = st["op"]
    if op == "ln_fwd":
        y, mean, rstd = jg.layernorm_fwd(st["x"], st["w"], st["b"], EPS, out_dtype=st["y_dtype"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dw, db = jg.layernorm_bwd(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], residual=st["res"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "ce_fwd":
        loss, lse = jg.linear_ce_fwd(st["x"], st["w"], st["b"], st["labels"], ignore_index=IGNORE,
                                     smoothing=st["smooth"])
        return {"loss": loss, "lse": lse}
    if op == "ce_bwd":
        dx, dw, db = jg.linear_ce_bwd(st["dloss"], st["x"], st["w"], st["b"], st["labels"], st["lse"],
                                      ignore_index=IGNORE, smoothing=st["smooth"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "ffn_fwd":
        return jg.gated_ffn_fwd(st["x"], st["wg"], st["wu"], st["bg"], st["bu"], act=st["act"])
    if op == "ffn_bwd":
        dx, dwg, dwu, dbg, dbu = jg.gated_ffn_bwd(st["dh"], st["x"], st["wg"], st["wu"], st["bg"], st["bu"],
                                                  act=st["act"])
        out = {"dx": dx, "dwg": dwg, "dwu": dwu}
        if st["bg"] is not None:
            out["dbg"], out["dbu"] = dbg, dbu
        return out
    da, dw, db = jg.linear_bwd(st["dy"], st["a"], st["w"], bias=st["bias"])
    return {"da": da, "dw": dw, "db": db} if st["bias"] else {"da": da, "dw": dw}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    op, m = case["op"], case["rows"]
    if op.startswith("ln"):
        n, sx, sy = m * case["dim"], size[case["x"]], size[case["y"]]
        if op == "ln_fwd":
            return {"bytes": n * (sx + sy) + 8 * m + 8 * case["dim"], "flops": 8 * n}
        res = sx if case["res"] else 0
        return {"bytes": n * (sx + sy + sx + res) + 8 * m + 12 * case["dim"], "flops": 16 * n}
    s = size[case["dtype"]]
    if op.startswith("ce"):
        d, v = case["dim"], case["vocab"]
        ins = s * (m * d + v * d) + 4 * v + 8 * m
        if op == "ce_fwd":
            return {"bytes": ins + 8 * m, "flops": 2 * m * d * v}
        return {"bytes": 2 * s * (m * d + v * d) + 8 * v + 16 * m, "flops": 6 * m * d * v}
    if op == "linear_bwd":
        n, k = case["n"], case["k"]
        return {"bytes": s * (2 * m * k + 2 * n * k + m * n) + (4 * n if case["bias"] else 0), "flops": 4 * m * n * k}
    d, f = case["dim"], case["hidden"]
    nb = 8 * f if case["bias"] else 0
    if op == "ffn_fwd":
        return {"bytes": s * (m * d + 2 * f * d + m * f) + nb, "flops": 4 * m * d * f}
    return {"bytes": s * (2 * m * d + 4 * f * d + m * f) + 2 * nb, "flops": 12 * m * d * f}


# ----------------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    """The outputs of ``run`` from the definitions in 64 bits, rows in pieces."""
    if work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    op, rows = st["op"], case["rows"]
    d = {k: (v.double() if torch.is_tensor(v) and v.is_floating_point() else v) for k, v in st.items()
         if k not in ("x", "dy", "res", "dh", "a")}

    def pieces(width):
        step = max(1, (1 << 28) // max(width, 1))
        return [slice(i, min(i + step, rows)) for i in range(0, rows, step)]

    def add(total, part):
        return part if total is None else total.add_(part)

    if op == "ln_fwd":
        parts = []
        for s in pieces(case["dim"]):
            x = st["x"][s].double()
            mu = x.sum(1) / x.shape[1]
            dev = x - mu.unsqueeze(1)
            rs = torch.rsqrt((dev * dev).sum(1) / x.shape[1] + EPS)
            parts.append((dev * rs.unsqueeze(1) * d["w"].unsqueeze(0) + d["b"].unsqueeze(0), mu, rs))
        y, mu, rs = (torch.cat(t) for t in zip(*parts))
        return {"y": y, "mean": mu, "rstd": rs}
    if op == "ln_bwd":
        dxs, dw, db = [], None, None
        for s in pieces(case["dim"]):
            x, dy = st["x"][s].double(), st["dy"][s].double()
            n = x.shape[1]
            r = d["rstd"][s].unsqueeze(1)
            xn = (x - d["mean"][s].unsqueeze(1)) * r
            wdy = dy * d["w"].unsqueeze(0)
            # y_i = w_i xn_i + b_i; d xn_j / d x_i = r (delta_ij - 1/n - xn_i xn_j / n)
            dx = (wdy - wdy.sum(1, keepdim=True) / n - xn * (wdy * xn).sum(1, keepdim=True) / n) * r
            if st["res"] is not None:
                dx = dx + st["res"][s].double()
            dxs.append(dx)
            dw, db = add(dw, (dy * xn).sum(0)), add(db, dy.sum(0))
        return {"dx": torch.cat(dxs), "dw": dw, "db": db}
    if op.startswith("ce"):
        v, sm = case["vocab"], case["smooth"]
        loss, lses, dxs, dw, db = [], [], [], None, None
        for s in pieces(v):
            x, lab = st["x"][s].double(), st["labels"][s]
            z = torch.addmm(d["b"].unsqueeze(0), x, d["w"].t())
            keep = lab.ne(IGNORE)
            target = torch.full_like(z, sm / v)
            target[torch.arange(len(lab), device=z.device)[keep], lab[keep]] += 1.0 - sm
            if op == "ce_fwd":
                lse = torch.logsumexp(z, 1)
                loss.append(torch.where(keep, lse - (target * z).sum(1), torch.zeros_like(lse)))
                lses.append(lse)
                continue
            dz = torch.exp(z - d["lse"][s].unsqueeze(1))
            dz = (dz - target) * (d["dloss"][s] * keep).unsqueeze(1)
            dxs.append(dz.mm(d["w"]))
            dw, db = add(dw, dz.t().mm(x)), add(db, dz.sum(0))
        if op == "ce_fwd":
            return {"loss": torch.cat(loss), "lse": torch.cat(lses)}
        return {"dx": torch.cat(dxs), "dw": dw, "db": db}
    if op == "linear_bwd":
        dy, a = st["dy"].double(), st["a"].double()
        out = {"da": dy.mm(d["w"]), "dw": dy.t().mm(a)}
        if st["bias"]:
            out["db"] = dy.sum(0)
        return out
    hs, dxs, tot = [], [], {}
    for s in pieces(2 * case["hidden"]):
        x = st["x"][s].double()
        gate, up = x.mm(d["wg"].t()), x.mm(d["wu"].t())
        if d["bg"] is not None:
            gate, up = gate + d["bg"].unsqueeze(0), up + d["bu"].unsqueeze(0)
        if case["act"] == "silu":
            sig = torch.sigmoid(gate)
            a, da = gate * sig, sig + gate * sig * (1.0 - sig)
        else:
            cdf = 0.5 * torch.erfc(-gate / math.sqrt(2.0))
            a, da = gate * cdf, cdf + gate * torch.exp(-gate * gate / 2.0) / math.sqrt(2.0 * math.pi)
        if op == "ffn_fwd":
            hs.append(a * up)
            continue
        dh = st["dh"][s].double()
        dgate, dup = dh * up * da, dh * a
        dxs.append(dgate.mm(d["wg"]) + dup.mm(d["wu"]))
        for k, part in (("dwg", dgate.t().mm(x)), ("dwu", dup.t().mm(x)), ("dbg", dgate.sum(0)), ("dbu", dup.sum(0))):
            tot[k] = add(tot.get(k), part)
    if op == "ffn_fwd":
        return torch.cat(hs)
    out = {"dx": torch.cat(dxs), "dwg": tot["dwg"], "dwu": tot["dwu"]}
    if st["bg"] is not None:
        out["dbg"], out["dbu"] = tot["dbg"], tot["dbu"]
    return out
