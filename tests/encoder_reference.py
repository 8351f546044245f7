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
