"""Plain float64 forms of the encoder-layer training operators, with bounds on
what a kernel's roundings may add to them (elementwise, derived from the
formulas).  No code of the package is used."""
from __future__ import annotations

import math

U32 = 2.0 ** -24          # half a step of float32
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step of the tensors' type


def buckets(len_q, len_k, borders, two_sided):
    import torch
    i = torch.arange(len_q)[:, None] + (len_k - len_q)
    j = torch.arange(len_k)[None, :]
    dist = (j - i).abs() if two_sided else (i - j).clamp_min(0)
    n = torch.zeros(len_q, len_k, dtype=torch.int64)
    for b in borders:
        n += dist >= b
    if two_sided:
        n += (j > i) * (len(borders) + 1)
    return n


def attention(q, k, v, scale, causal=False, lens=None, bias=None, borders=(), two_sided=True, out=None, lse=None,
              dout=None, dtype="f32", roundings=16):
    """Values and error bounds, {name: (value, bound)}.  All inputs are CPU
    tensors; with dout the gradients, from the given out and lse, else out and
    lse.  `roundings`: how often a score may be rounded at its own size."""
    import torch
    B, Lq, H, D = q.shape
    Lk, Hk = k.shape[1], k.shape[2]
    g = H // Hk
    qd, kd, vd = (t.double().permute(0, 2, 1, 3) for t in (q, k, v))
    see = torch.ones(B, 1, Lq, Lk, dtype=torch.bool)
    j = torch.arange(Lk)
    if lens is not None:
        see = see & (j < lens.long()[:, None, None, None])
        # hidden keys may hold anything
        hid = (j[None, None, :, None] >= lens.long()[:, None, None, None])
        kd = torch.where(hid, torch.zeros_like(kd), kd)
        vd = torch.where(hid, torch.zeros_like(vd), vd)
    if causal:
        see = see & (j <= torch.arange(Lq)[:, None] + (Lk - Lq))
    kr, vr = kd.repeat_interleave(g, 1), vd.repeat_interleave(g, 1)
    s = qd @ kr.transpose(2, 3) * scale
    bk = None
    if bias is not None:
        bk = buckets(Lq, Lk, borders, two_sided)
        s = s + bias.double().t()[:, bk]
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    rnd = HALF[dtype]
    low = 0.0 if dtype == "f32" else rnd      # rounding of P and dS into their products
    # relative error of a probability: the score's sum of D products, its
    # additions, the logarithm's, and the exponential's
    sizes = (qd.abs() @ kr.abs().transpose(2, 3)) * scale
    ep = U32 * ((D + 4) * sizes + roundings * (torch.where(see, s, torch.zeros_like(s)).abs() + 8)) + 8 * U32
    res = {}
    if dout is None:
        m = s.amax(dim=3, keepdim=True) if Lk else torch.full((B, H, Lq, 1), -math.inf, dtype=torch.float64)
        m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        e = torch.exp(s - m0)
        z = e.sum(3, keepdim=True)
        p = e / torch.where(z > 0, z, torch.ones_like(z))
        o = p @ vr
        row = (p * ep).sum(3, keepdim=True)       # the sum's relative error, in every probability of the row
        err = (p * (ep + row + low + (Lk + 8) * U32)) @ vr.abs()
        res["out"] = (o.permute(0, 2, 1, 3), (err + rnd * o.abs()).permute(0, 2, 1, 3))
        l = (m0 + torch.log(z)).squeeze(3)
        res["lse"] = (l, row.squeeze(3) + (Lk + 8) * U32 + 4 * U32 * l.abs().nan_to_num(posinf=0.0))
        return res
    L = lse.double()[..., None]
    p = torch.where(see, torch.exp(s - torch.where(torch.isinf(L), torch.zeros_like(L), L)), torch.zeros_like(s))
    do, od = dout.double().permute(0, 2, 1, 3), out.double().permute(0, 2, 1, 3)
    delta = (do * od).sum(3, keepdim=True)
    dp = do @ vr.transpose(2, 3)
    ds = p * (dp - delta)
    eds = ep * ds.abs() + (D + 4) * U32 * p * (do.abs() @ vr.abs().transpose(2, 3) + (do * od).abs().sum(3, keepdim=True))

    def fold(x):
        return x.reshape(B, Hk, g, Lk, D).sum(2).permute(0, 2, 1, 3)

    def bound(value, left, eleft, right, n):
        return (eleft + (low + n * U32) * left.abs()) @ right.abs()

    dq = ds @ kr * scale
    res["dq"] = (dq.permute(0, 2, 1, 3), (bound(dq, ds, eds, kr, Lk + 8) * scale + rnd * dq.abs()).permute(0, 2, 1, 3))
    dst, edst, pt = ds.transpose(2, 3), eds.transpose(2, 3), p.transpose(2, 3)
    dk = fold(dst @ qd * scale)
    res["dk"] = (dk, fold(bound(dk, dst, edst, qd, g * Lq + 8) * scale) + rnd * dk.abs())
    dv = fold(pt @ do)
    res["dv"] = (dv, fold(bound(dv, pt, (ep * p).transpose(2, 3), do, g * Lq + 8)) + rnd * dv.abs())
    if bias is not None:
        n = bias.shape[0]
        val, err = torch.zeros(n, H, dtype=torch.float64), torch.zeros(n, H, dtype=torch.float64)
        terms = B * Lq * Lk
        for b in range(n):
            at = (bk == b).double()
            val[b] = (ds * at).sum((0, 2, 3))
            err[b] = ((eds + (min(terms, 4096) + 8) * U32 * ds.abs()) * at).sum((0, 2, 3))
        res["dbias"] = (val, err)
    return res


# ------------------------------------------------------------- checkpoints --

def encode(x, ones):
    """codes [blocks, d, 32] and scales [blocks, d] of x [rows, d] (numpy, float64 arithmetic)."""
    import numpy as np
    x = np.asarray(x, dtype=np.float64)
    if ones:
        x = np.concatenate([x, np.ones((x.shape[0], 1))], 1)
    rows, d = x.shape
    blocks = (rows + 31) // 32
    full = np.zeros((blocks * 32, d))
    full[:rows] = x
    full = full.reshape(blocks, 32, d).transpose(0, 2, 1)
    fin = np.where(np.isfinite(full), np.abs(full), 0.0)
    top = fin.max(axis=2)
    e = np.full(top.shape, -117, dtype=np.int64)
    for n in range(-117, 125):
        e = np.where(top > 448.0 * 2.0 ** n, n + 1, e)
    y = np.abs(full) / (2.0 ** e)[:, :, None]
    with np.errstate(invalid="ignore"):
        _, ex = np.frexp(np.where(np.isfinite(y), y, 0.0))
        ex = np.maximum(ex - 1, -6)
        step = 2.0 ** (ex - 3)
        q = np.rint(np.where(np.isfinite(y), y, 0.0) / step)      # multiples of the step, ties to even
    v = q * step
    _, ev = np.frexp(v)
    ev = np.maximum(ev - 1, -6)
    m = np.rint(v / 2.0 ** (ev - 3)).astype(np.int64)               # 8 .. 15, or 0 .. 7 where the exponent is least
    code = np.where(m >= 8, ((ev + 7) << 3) + (m - 8), m)
    code = np.where(np.isfinite(full), code, 0x7f)
    sign = np.signbit(full) & ~np.isnan(full)
    return (code | (sign.astype(np.int64) << 7)).astype(np.uint8), (e + 127).astype(np.uint8)


def decode(codes, scales, rows):
    import numpy as np
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7).astype(np.float64))
    v = np.where((c & 0x7f) == 0x7f, np.nan, v) * np.where(c >> 7, -1.0, 1.0)
    v = v * 2.0 ** (scales.astype(np.float64) - 127)[:, :, None]
    return v.transpose(0, 2, 1).reshape(-1, codes.shape[1])[:rows]
