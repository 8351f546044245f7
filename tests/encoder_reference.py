"""Plain float64 forms of layer norm and of gradient clipping, with bounds on
what a kernel's roundings may add (elementwise, to first order, from the
formulas).  No code of the package is used."""
from __future__ import annotations

U32 = 2.0 ** -24                                # half a step of float32
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step of a type
# additions behind one another in a row's sum: 16 elements of a lane, 6 steps over a wave, 16 waves
DEPTH = 48


def types():
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}


def norm_forward(x, weight, bias, eps, dtype):
    """{name: (value, bound)} of y, mean, rstd."""
    import torch
    x = x.double()
    d = x.shape[1]
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(d, dtype=torch.float64) if bias is None else bias.double()
    mean = x.mean(1, keepdim=True)
    e_mean = (DEPTH + 3) * U32 * x.abs().mean(1, keepdim=True)     # the sum, 1 / d and the product with it
    c = x - mean
    e_c = e_mean + U32 * c.abs()
    var = c.square().mean(1, keepdim=True)
    # sum (c - e)^2 = sum c^2 + d e^2 for an error e that all elements share
    e_var = (DEPTH + 8) * U32 * var + e_mean.square()
    rstd = (var + eps) ** -0.5
    rel = 0.5 * e_var / (var + eps) + 4 * U32
    y = c * rstd * w + b
    e_y = w.abs() * (rstd * e_c + (c * rstd).abs() * (rel + 3 * U32)) + (U32 + HALF[dtype]) * (y.abs() + b.abs())
    return {"y": (y, e_y), "mean": (mean[:, 0], e_mean[:, 0]), "rstd": (rstd[:, 0], (rel * rstd)[:, 0])}


def norm_backward(dy, x, mean, rstd, weight, dtype, weight_dtype):
    """{name: (value, bound)} of dx, dweight, dbias, from the statistics as they are."""
    import torch
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, d = x.shape
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    xh = (x - mean) * rstd                                          # 2 roundings
    a = dy * w                                                      # 1
    m0, m1 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    e0 = (DEPTH + 4) * U32 * a.abs().mean(1, keepdim=True)
    e1 = (DEPTH + 8) * U32 * (a * xh).abs().mean(1, keepdim=True)
    dx = rstd * (a - m0 - xh * m1)
    e_dx = rstd * (e0 + xh.abs() * e1 + 8 * U32 * (a.abs() + m0.abs() + (xh * m1).abs())) + HALF[dtype] * dx.abs()
    # a wave's rows, four waves, 32 workgroups' sums in turn, 16 groups
    depth = rows // 512 + 1 + 4 + 32 + 16
    low = 0.0 if weight_dtype == "f32" else HALF[weight_dtype]
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return {"dx": (dx, e_dx), "dweight": (dw, (depth + 4) * U32 * (dy * xh).abs().sum(0) + low * dw.abs()),
            "dbias": (db, depth * U32 * dy.abs().sum(0) + low * db.abs())}


def worst(got, value, bound):
    """The largest error in units of its bound (0 / 0 counts as 0)."""
    import torch
    err = (got.double().cpu() - value).abs()
    if err.numel() == 0:
        return 0.0
    ratio = torch.where(err > 0, err / bound.clamp_min(1e-300), torch.zeros_like(err))
    return float(ratio.nan_to_num(nan=float("inf")).max())


# ------------------------------------------------------------------- gated --

def activation(name, g):
    """(act, its slope, bounds on what a float32 evaluation may be off by), float64."""
    import math

    import torch
    if name == "relu":
        a, q, rest = g.clamp_min(0), (g > 0).double(), torch.zeros_like(g)
    elif name in ("silu", "sigmoid"):
        s = torch.sigmoid(g)
        t = s * torch.sigmoid(-g)
        a, q, rest = (s, t, torch.zeros_like(g)) if name == "sigmoid" else (g * s, s, g * t)
    elif name == "gelu":
        q = 0.5 * torch.erfc(-g / math.sqrt(2))
        a, rest = g * q, g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        c = math.sqrt(8 / math.pi)
        z = c * (g + 0.044715 * g ** 3)
        q = torch.sigmoid(z)
        a, rest = g * q, g * q * torch.sigmoid(-z) * c * (1 + 0.134145 * g * g)
    # functions of some roundings, and an exponent's relative error: its
    # argument's, g^2 / 2 or 1.6 |g| + 0.07 |g|^3, times that argument
    rel = (16 + 8 * g.abs() + 4 * g * g + g.abs() ** 3) * U32
    return a, q + rest, rel * a.abs(), rel * (q.abs() + rest.abs())


def product(a, b, dtype):
    """a b and the bound of its float32 sum: each of the K additions rounds,
    and float32 products lose the parts' last cross terms, 2.01 steps."""
    return a @ b, (1.05 * a.shape[1] + 12) * U32 * (a.abs() @ b.abs())


def gated_forward(x, weight, bias, act, dtype):
    import torch
    x, w = x.double(), weight.double()
    n = w.shape[0] // 2
    pre, e = product(x, w.t(), dtype)
    if bias is not None:
        pre = pre + bias.double()
        e = e + U32 * pre.abs()
    a, slope, e_a, _ = activation(act, pre[:, :n])
    h = a * pre[:, n:]
    e_h = (e_a + 1.2 * e[:, :n]) * (pre[:, n:].abs() + e[:, n:]) + a.abs() * e[:, n:] + U32 * h.abs()
    return {"h": (h, e_h + HALF[dtype] * h.abs()), "pre": (pre, e + HALF[dtype] * pre.abs())}


def gated_backward(dh, x, weight, pre, dpre, act, dtype, dweight_dtype):
    """dpre and dbias from the inputs; dx and dweight from dpre as it was given out."""
    import torch
    n = weight.shape[0] // 2
    dh, g, u = dh.double(), pre.double()[:, :n], pre.double()[:, n:]
    a, slope, e_a, e_s = activation(act, g)
    dg, du = dh * u * slope, dh * a
    want = torch.cat([dg, du], 1)
    e = torch.cat([(dh * u).abs() * e_s + 3 * U32 * dg.abs(), dh.abs() * e_a + 2 * U32 * du.abs()], 1)
    # Relative steps end at the least normal number, 2^-126: below it a
    # bfloat16 result is off by up to half of 2^-133, a float32 one by half of
    # 2^-149, and so is each of a term's dozen float32 products on the way,
    # which the later factors (g, 1 + 0.134 g^2, dh u) multiply.  (A value of
    # -2.2e-41 has no nearer bfloat16 number than 0: 2.2e-41 <= 2^-134.)
    small = 12 * 2.0 ** -150 * (1 + g.abs() + g.abs() ** 3) * (1 + dh.abs() * (1 + u.abs()))
    e = e + torch.cat([small, small], 1) + (2.0 ** -134 if dtype == "bf16" else 2.0 ** -150)
    res = {"dpre": (want, e + HALF[dtype] * want.abs())}
    # a wave's rows of a chunk, four waves, 32 chunks in turn, 16 groups
    depth = dh.shape[0] + 64
    res["dbias"] = (want.sum(0), e.sum(0) + depth * U32 * want.abs().sum(0))
    p = dpre.double()
    dx, e = product(p, weight.double(), dtype)
    res["dx"] = (dx, e + HALF[dtype] * dx.abs())
    dw, e = product(p.t(), x.double(), dtype)
    res["dweight"] = (dw, e + HALF[dweight_dtype] * dw.abs())
    return res
