"""The rest of an encoder's training step under the preconditioner: what is
measured, in plain torch operations and through the package.

    layer norm forward / backward   rows normalised to mean 0 and variance 1,
                                    scaled and shifted; gradients of the input,
                                    of the scale and of the shift
    gated forward / backward        [g | u] = x W^T + b, h = act(g) u; gradients
                                    of [g | u], of x, of W and of b
    clip                            the norm of many gradients taken together,
                                    and the gradients scaled down to a norm
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


# ------------------------------------------------------------------ cases --

def _norm(name, op, dtype, rows, d):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "d": d}


def _gated(name, op, dtype, rows, d, width, act, keep=True):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "d": d, "width": width, "act": act, "keep": keep}


def listed():
    return [
        # one short sequence of the encoder's width: what a call costs
        _norm("norm_fwd_short", "norm_fwd", "bf16", 77, 1024),
        # the encoder's layer: 4096 tokens of width 1024
        _norm("norm_fwd_encoder", "norm_fwd", "bf16", 4096, 1024),
        _norm("norm_bwd_encoder", "norm_bwd", "bf16", 4096, 1024),
        # float32 with an odd width, at the rows of the largest workload
        _norm("norm_bwd_odd", "norm_bwd", "f32", 25088, 2305),
        # the gradients of one small layer, of a ResNet-50 (matrices in bfloat16, vectors in float32), of the 12-layer encoder
        {"name": "clip_fc", "op": "clip", "dtype": "f32", "set": "fc"},
        {"name": "clip_resnet50", "op": "clip", "dtype": "mixed", "set": "resnet50"},
        {"name": "clip_encoder", "op": "clip", "dtype": "f32", "set": "encoder"},
        # a single token through the encoder's feed-forward width, nothing kept for a backward pass
        _gated("gated_fwd_token", "gated_fwd", "bf16", 1, 1024, 4096, "silu", keep=False),
        # training the encoder's block: two thirds of 4096 wide, which gives the three matrices a plain block's weights
        _gated("gated_fwd_encoder", "gated_fwd", "bf16", 4096, 1024, 2730, "gelu"),
        _gated("gated_bwd_encoder", "gated_bwd", "bf16", 4096, 1024, 2730, "gelu"),
        # float32 with odd sizes
        _gated("gated_bwd_odd_f32", "gated_bwd", "f32", 333, 1001, 1365, "gelu_tanh"),
        # the rows and widths of the largest workload
        _gated("gated_bwd_large", "gated_bwd", "bf16", 25088, 2304, 4608, "silu"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Sizes over the listed cases' ranges, redrawn until the work is at most the largest listed case's."""
    while True:
        op = rng.choice(("norm_fwd", "norm_bwd", "clip", "gated_fwd", "gated_bwd", "gated_bwd"))
        dtype = rng.choice(("bf16", "f32"))
        if op.startswith("norm"):
            # rows of a few elements have gradients that are zero but for rounding, which leaves nothing to compare
            case = {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 25088), "d": _log_int(rng, 16, 8192)}
            if case["rows"] * case["d"] > 25088 * 2305:
                continue
        elif op == "clip":
            most = _log_int(rng, 16, 4 << 20)
            case = {"op": op, "dtype": rng.choice(("bf16", "f32", "mixed")), "set": "spread", "tensors": _log_int(rng, 1, 400),
                    "most": most, "order": rng.randrange(1 << 20), "share": rng.choice((0.01, 0.5, 2.0))}
            if sum(_sizes(case)) > 150e6:
                continue
        else:
            case = {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 25088), "d": _log_int(rng, 16, 4608),
                    "width": _log_int(rng, 32, 5460), "act": rng.choice(ACTS), "keep": op == "gated_bwd" or rng.random() < 0.5}
            if work(case)["flops"] > (2e12 if dtype == "bf16" else 2.5e11):
                continue
        return case


def _sizes(case):
    """Elements of each gradient of a set, vectors (biases, scales) among the matrices."""
    if case["set"] == "fc":
        return [32 * 64, 32]
    if case["set"] == "encoder":
        w = 1024
        return [n for _ in range(12) for n in (w, w, 3 * w * w, 3 * w, w * w, w, w, w, 4 * w * w, 4 * w, 4 * w * w, w)]
    if case["set"] == "resnet50":
        got = [64 * 3 * 49, 64, 64]
        c_in = 64
        for blocks, width, out in ((3, 64, 256), (4, 128, 512), (6, 256, 1024), (3, 512, 2048)):
            for b in range(blocks):
                got += [c_in * width, width, width, 9 * width * width, width, width, width * out, out, out]
                if b == 0:
                    got += [c_in * out, out, out]
                c_in = out
        return got + [2048 * 1000, 1000]
    rng = random.Random(case["order"])
    return [_log_int(rng, 1, case["most"]) for _ in range(case["tensors"])]


def _is_bf16(case, size):
    """Which gradients are bfloat16: in a mixed set the larger ones."""
    return case["dtype"] == "bf16" or (case["dtype"] == "mixed" and size > 4096)


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(s * (2 if _is_bf16(case, s) else 4) for s in _sizes(case))
        return {"bytes": 2 * n + 4, "flops": 3 * sum(_sizes(case))}
    rows, d, es = case["rows"], case["d"], 2 if case["dtype"] == "bf16" else 4
    if op == "norm_fwd":
        return {"bytes": 2 * rows * d * es + 8 * rows + 8 * d, "flops": 8 * rows * d}
    if op == "norm_bwd":
        return {"bytes": 3 * rows * d * es + 8 * rows + 12 * d, "flops": 14 * rows * d}
    w = case["width"]
    if op == "gated_fwd":
        return {"bytes": (rows * d + 2 * w * d + rows * w * (3 if case["keep"] else 1)) * es + 8 * w, "flops": 4 * rows * d * w}
    return {"bytes": (2 * rows * d + 4 * w * d + 5 * rows * w) * es + 8 * w, "flops": 8 * rows * d * w}


# ----------------------------------------------------------------- inputs --

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _clip_state(case, g):
    """Gradients as views of one buffer for each type, as bucketed gradients lie, and room for the clipped ones."""
    s = {"case": case, "norm": torch.empty(1, device=DEV)}
    sizes = _sizes(case)
    views, total = [], 0.0
    for key, t in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        mine = [n for n in sizes if _is_bf16(case, n) == (key == "bf16")]
        if not mine:
            continue
        flat = torch.randn(sum(mine), device=DEV, generator=g)
        # layers' gradients differ in size
        for part in flat.split(mine):
            part.mul_(1e-3 * math.exp(2.0 * math.sin(len(views) + part.numel())))
            views.append(part)
        flat = flat.to(t)
        s[key], s["out_" + key] = flat, torch.empty_like(flat)
        total += float(flat.double().square().sum())
        views[-len(mine):] = zip(flat.split(mine), s["out_" + key].split(mine))
    s["grads"], s["outs"] = [list(v) for v in zip(*views)]
    # a tenth or half of the norm (clipped) or twice it (left as they are)
    s["max_norm"] = math.sqrt(total) * case.get("share", 0.1)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "clip":
        return _clip_state(case, g)
    t, rows, d = _type(case), case["rows"], case["d"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device=DEV, generator=g).mul_(std)

    s = {"case": case, "eps": 1e-5}
    if case["op"].startswith("norm"):
        # a residual stream: tokens of different size, a shift, a few columns much larger than the others
        x = normal(rows, d).mul_(torch.exp(0.5 * normal(rows, 1))).add_(0.2 * normal(rows, 1))
        x[:, torch.rand(d, device=DEV, generator=g) < 0.02] *= 20.0
        s["x"] = x.to(t)
        s["weight"], s["bias"] = 1.0 + normal(d, std=0.2), normal(d, std=0.1)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, d, std=0.02).to(t)
            s["mean"], s["rstd"] = _plain_stats(s)
        return s
    w = case["width"]
    s["x"] = normal(rows, d).to(t)
    s["weight"] = normal(2 * w, d, std=d ** -0.5).to(t)
    s["bias"] = normal(2 * w, std=0.1)
    if case["op"] == "gated_bwd":
        s["pre"] = (torch.matmul(s["x"].float(), s["weight"].float().t()) + s["bias"]).to(t)
        s["dh"] = normal(rows, w, std=0.02).to(t)
    return s


# ------------------------------------------------------------- plain forms --

def _plain_stats(s):
    x = s["x"].float()
    mean = x.mean(dim=1)
    return mean, torch.rsqrt((x - mean[:, None]).square().mean(dim=1) + s["eps"])


def _plain_norm(s):
    x, w = s["x"].float(), s["weight"]
    if s["case"]["op"] == "norm_fwd":
        mean, rstd = _plain_stats(s)
        y = (x - mean[:, None]) * rstd[:, None] * w + s["bias"]
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    rstd, dy = s["rstd"][:, None], s["dy"].float()
    xh = (x - s["mean"][:, None]) * rstd
    a = dy * w
    dx = rstd * (a - a.mean(dim=1, keepdim=True) - xh * (a * xh).mean(dim=1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(dim=0), "dbias": dy.sum(dim=0)}


def _plain_act(name, g):
    """act(g) and its derivative."""
    if name == "relu":
        return g.clamp_min(0), (g > 0).to(g.dtype)
    if name in ("silu", "sigmoid"):
        q = 1 / (1 + torch.exp(-g))
        return (q, q * (1 - q)) if name == "sigmoid" else (g * q, q * (1 + g * (1 - q)))
    if name == "gelu":
        q = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
        return g * q, q + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


def _plain_gated(s):
    c, t = s["case"], s["x"].dtype
    w, x, m = c["width"], s["x"].float(), s["weight"].float()
    if c["op"] == "gated_fwd":
        pre = torch.matmul(x, m.t()) + s["bias"]
        got = {"h": (_plain_act(c["act"], pre[:, :w])[0] * pre[:, w:]).to(t)}
        return dict(got, pre=pre.to(t)) if c["keep"] else got
    g, u, dh = s["pre"][:, :w].float(), s["pre"][:, w:].float(), s["dh"].float()
    a, da = _plain_act(c["act"], g)
    dpre = torch.cat([dh * u * da, dh * a], dim=1)
    return {"dpre": dpre.to(t), "dx": torch.matmul(dpre, m).to(t), "dweight": torch.matmul(dpre.t(), x).to(t),
            "dbias": dpre.sum(dim=0)}


def _plain_clip(s):
    total = sum(g.double().square().sum() for g in s["grads"])
    norm = torch.sqrt(total)
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
    got = {"norm": norm.float().reshape(1)}
    for key in ("bf16", "f32"):
        if key in s:
            got[key] = (s[key].float() * scale).to(s[key].dtype)
    return got


# ------------------------------------------------------------------ one pass --

def _own(s):
    import linear_algebra_amd as la

    c, op = s["case"], s["case"]["op"]
    if op == "clip":
        la.kfac_grad_clip(s["grads"], s["max_norm"], s["norm"], outs=s["outs"])
        return {"norm": s["norm"], **{k: s["out_" + k] for k in ("bf16", "f32") if k in s}}
    x = s["x"]
    if op == "norm_fwd":
        y, mean, rstd = torch.empty_like(x), torch.empty(c["rows"], device=DEV), torch.empty(c["rows"], device=DEV)
        la.kfac_layer_norm_forward(x, y, mean, rstd, weight=s["weight"], bias=s["bias"], eps=s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dw, db = torch.empty_like(x), torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
        la.kfac_layer_norm_backward(s["dy"], x, s["mean"], s["rstd"], dx, weight=s["weight"], dweight=dw, dbias=db)
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "gated_fwd":
        got = {"h": torch.empty(c["rows"], c["width"], dtype=x.dtype, device=DEV)}
        if c["keep"]:
            got["pre"] = torch.empty(c["rows"], 2 * c["width"], dtype=x.dtype, device=DEV)
        la.kfac_gated_forward(x, s["weight"], got["h"], bias=s["bias"], pre=got.get("pre"), activation=c["act"])
        return got
    got = {"dpre": torch.empty_like(s["pre"]), "dx": torch.empty_like(x), "dweight": torch.empty_like(s["weight"]),
           "dbias": torch.empty_like(s["bias"])}
    la.kfac_gated_backward(s["dh"], x, s["weight"], s["pre"], activation=c["act"], **got)
    return got


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_clip(state) if op == "clip" else _plain_norm(state) if op.startswith("norm") else _plain_gated(state)


# ------------------------------------------------------------------- 64 bits --

def _exact_act(name, g):
    """act(g) and its derivative, by other ways to the same functions."""
    if name == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g)), torch.where(g > 0, torch.ones_like(g), torch.zeros_like(g))
    if name in ("silu", "sigmoid"):
        q = torch.sigmoid(g)
        slope = q * torch.sigmoid(-g)
        return (q, slope) if name == "sigmoid" else (g * q, q + g * slope)
    if name == "gelu":
        q = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * q, q + g * torch.exp(-(g ** 2) / 2) / math.sqrt(2 * math.pi)
    # (1 + tanh z) / 2 = sigmoid(2 z)
    z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    q = torch.sigmoid(z)
    return g * q, q + g * q * torch.sigmoid(-z) * math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(s[k].double().square().sum()) for k in ("bf16", "f32") if k in s))
        scale = min(1.0, s["max_norm"] / (norm + 1e-6))
        got = {k: s[k].double() * scale for k in ("bf16", "f32") if k in s}
        return {"norm": torch.tensor([norm], dtype=torch.float64, device=DEV), **got}
    x, w = s["x"].double(), s["weight"].double()
    if case["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + s["eps"]) ** -0.5
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w)
        return {"y": y, "mean": mean, "rstd": rstd}
    if case["op"] == "norm_bwd":
        n, dy, r = case["d"], s["dy"].double(), s["rstd"].double()[:, None]
        xh = (x - s["mean"].double()[:, None]) * r
        along, across = dy @ w / n, (dy * xh) @ w / n
        dx = r * (dy * w - along[:, None] - xh * across[:, None])
        return {"dx": dx, "dweight": torch.einsum("ij,ij->j", dy, xh), "dbias": dy.sum(dim=0)}
    n = case["width"]
    if case["op"] == "gated_fwd":
        gate = torch.addmm(s["bias"][:n].double(), x, w[:n].t())
        up = torch.addmm(s["bias"][n:].double(), x, w[n:].t())
        h = _exact_act(case["act"], gate)[0] * up
        return {"h": h, "pre": torch.cat([gate, up], dim=1)} if case["keep"] else {"h": h}
    gate, up, dh = s["pre"][:, :n].double(), s["pre"][:, n:].double(), s["dh"].double()
    a, slope = _exact_act(case["act"], gate)
    dgate, dup = dh * up * slope, dh * a
    return {"dpre": torch.cat([dgate, dup], dim=1), "dx": dgate @ w[:n] + dup @ w[n:],
            "dweight": torch.cat([dgate.t() @ x, dup.t() @ x]), "dbias": torch.cat([dgate.sum(0), dup.sum(0)])}
