"""The operators that train an encoder layer under the preconditioner: what is
measured, in plain torch operations and through the package.

    attention forward / backward   softmax attention with a learned relative
                                   position bias by buckets; the backward pass
                                   recomputes the probabilities from lse
    checkpoint round trip          a layer input kept in 8 bits, and read back
    checkpoint factor              A = x^T x / rows from the kept input
    checkpoint gradient            [dW | db] = g^T [x | 1] from the kept input

A kept input holds blocks of 32 consecutive rows of one column: e4m3 codes
[blocks, columns, 32] and one power of two per block, its exponent plus 127,
[blocks, columns].  The exponent is the least one, not under -117, for which
the block's largest magnitude stays within 448 times the power.
"""
import math

import torch

own = False

DEV = "cuda:0"
E4M3_MAX = 448.0
MIN_EXP = -117


# ------------------------------------------------------------------ cases --

def _attn(name, op, dtype, batch, len_q, len_k, heads, kv_heads, dim, causal, buckets, far, fill):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "len_q": len_q, "len_k": len_k, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "causal": causal, "buckets": buckets, "far": far, "fill": fill}


def listed():
    return [
        # one short sequence: what a call costs when there is next to nothing to compute
        _attn("fwd_short", "attn_fwd", "bf16", 1, 77, 77, 4, 4, 32, False, 16, 128, 1.0),
        # the encoder's layer: 4096 tokens of width 1024 in sequences of uneven length, one slot empty
        _attn("fwd_encoder", "attn_fwd", "bf16", 8, 512, 512, 16, 16, 64, False, 16, 128, 0.0),
        # one long document, causal, heads that share keys and values
        _attn("fwd_long", "attn_fwd", "bf16", 1, 8192, 8192, 16, 4, 128, True, 32, 1024, 1.0),
        # float32 training with odd sizes: a head width that fills no tile, queries and keys of different lengths
        _attn("bwd_odd_f32", "attn_bwd", "f32", 3, 333, 401, 6, 3, 72, False, 12, 100, 0.5),
        _attn("bwd_encoder", "attn_bwd", "bf16", 8, 512, 512, 16, 16, 64, False, 16, 128, 0.0),
        _attn("bwd_long", "attn_bwd", "bf16", 1, 8192, 8192, 16, 4, 128, True, 32, 1024, 1.0),
        # the MLP's first layer: batch 128 of 1024 inputs, float32, with the column of ones
        {"name": "keep_mlp", "op": "keep", "dtype": "f32", "rows": 128, "d": 1024, "ones": True},
        # the encoder's second feed-forward layer: 4096 tokens of 4096 inputs
        {"name": "keep_ffn", "op": "keep", "dtype": "bf16", "rows": 4096, "d": 4096, "ones": True},
        # factors of the encoder's layers: inputs of 1024 and 4096 with the column of ones
        {"name": "factor_qkv", "op": "factor", "rows": 4096, "d": 1024, "ones": True},
        {"name": "factor_ffn", "op": "factor", "rows": 4096, "d": 4096, "ones": True},
        # gradients of an MLP layer in float32 and of the encoder's second feed-forward layer in bfloat16
        {"name": "grad_mlp_f32", "op": "grad", "dtype": "f32", "rows": 128, "d": 2048, "d_out": 1024, "ones": True},
        {"name": "grad_ffn", "op": "grad", "dtype": "bf16", "rows": 4096, "d": 4096, "d_out": 1024, "ones": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Sizes over the listed cases' ranges, redrawn until the work is at most the largest listed case's."""
    while True:
        op = rng.choice(("attn_fwd", "attn_bwd", "attn_bwd", "keep", "factor", "grad"))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        if op.startswith("attn"):
            causal = rng.random() < 0.5
            # through a single key the scores' gradients are zero but for rounding, which leaves nothing to compare
            least = 1 if op == "attn_fwd" else 8
            len_q = _log_int(rng, least, 8192)
            len_k = len_q if causal or rng.random() < 0.6 else _log_int(rng, least, 4096)
            batch = _log_int(rng, 1, 16)
            kv_heads = rng.choice((1, 2, 3, 4, 8, 16))
            heads = kv_heads * rng.choice((1, 1, 2, 3, 4))
            case = _attn("", op, dtype, batch, len_q, len_k, heads, kv_heads, 8 * rng.randint(2, 16), causal,
                         rng.choice((0, 8, 16, 24, 32)), rng.choice((64, 100, 128, 256, 1024)),
                         rng.choice((1.0, 0.5, 0.0)) if batch > 1 else 1.0)
            # the plain float32 form of a long case is the slow one: float32 draws stay at a sixteenth of the work
            most = 7e11 if dtype == "bf16" else 4.4e10
            pairs = case["batch"] * heads * len_q * len_k
            if heads > 24 or pairs > 1.1e9 or work(case)["flops"] > most:
                continue
        elif op == "keep":
            case = {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 25088), "d": _log_int(rng, 16, 4608),
                    "ones": rng.random() < 0.7}
            if case["rows"] * case["d"] > 4096 * 4097:
                continue
        elif op == "factor":
            case = {"op": op, "rows": _log_int(rng, 1, 25088), "d": _log_int(rng, 16, 4608), "ones": rng.random() < 0.7}
            if work(case)["flops"] > 7e10:
                continue
        else:
            case = {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 25088), "d": _log_int(rng, 16, 4608),
                    "d_out": _log_int(rng, 10, 4096), "ones": rng.random() < 0.7}
            if work(case)["flops"] > 7e10:
                continue
        case.pop("name", None)
        return case


def _lens(case):
    """Visible keys of each sequence: from fill * len_k to len_k in even steps (fill 1: all of them; 0: one is empty)."""
    n, lk = case["batch"], case["len_k"]
    if case["fill"] >= 1.0:
        return [lk] * n
    return [int(round(lk * (case["fill"] + (1.0 - case["fill"]) * i / max(1, n - 1)))) for i in range(n)]


def work(case):
    op = case["op"]
    if op.startswith("attn"):
        es = 2 if case["dtype"] == "bf16" else 4
        lq, lk, h, hk, d, b = (case[k] for k in ("len_q", "len_k", "heads", "kv_heads", "dim", "batch"))
        pairs = 0
        for n in _lens(case):
            if case["causal"]:
                # query i sees min(n, i + lk - lq + 1) keys
                first = lk - lq + 1
                full = max(0, min(lq, lq - max(0, n - first)))          # queries that see all n keys
                part = lq - full
                lo = max(0, first)
                skip = max(0, -first)
                part = max(0, part - skip)
                pairs += full * n + part * (2 * lo + part - 1) // 2
            else:
                pairs += lq * n
        pairs *= h
        qb, kb, lb = b * lq * h * d * es, b * sum(_lens(case)) // max(1, b) * hk * d * es, b * lq * h * 4
        table = case["buckets"] * h * 4
        if op == "attn_fwd":
            return {"bytes": 2 * qb + 2 * kb + lb + table, "flops": 4 * d * pairs}
        return {"bytes": 4 * qb + 4 * kb + lb + 2 * table, "flops": 10 * d * pairs}
    rows, da = case["rows"], case["d"] + int(case["ones"])
    codes = (rows + 31) // 32 * 33 * da
    if op == "keep":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * case["d"] * es + 2 * codes + rows * da * es, "flops": 0}
    if op == "factor":
        return {"bytes": codes + 2 * da * (da + 1), "flops": rows * da * (da + 1)}
    es = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": codes + rows * case["d_out"] * es + 4 * case["d_out"] * da, "flops": 2 * rows * case["d_out"] * da}


# ----------------------------------------------------------------- inputs --

def _type(case):
    return torch.bfloat16 if case.get("dtype") == "bf16" else torch.float32


def _borders(buckets, far, two_sided):
    """Where the buckets of one side begin: half of them single distances, the rest spread over the logarithm up to `far`.
    Whole-number comparisons, so that no distance lies on a rounded border."""
    n = buckets // 2 if two_sided else buckets
    near = n // 2
    got = list(range(1, near + 1))
    wide = n - near
    for m in range(1, wide):
        # the least t with (t / near)^wide >= (far / near)^m
        t = int(near * (far / near) ** (m / wide)) - 2
        t = max(t, got[-1])
        while t ** wide * near ** m < far ** m * near ** wide:
            t += 1
        got.append(max(t, got[-1] + 1))
    return got


def _attn_state(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = _type(case)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device=DEV, generator=g) * std).to(t)

    b, lq, lk, h, hk, d = (case[k] for k in ("batch", "len_q", "len_k", "heads", "kv_heads", "dim"))
    s = {"case": case, "scale": d ** -0.5, "two_sided": not case["causal"]}
    if lq == lk:
        # one projection's output holds queries, keys and values side by side
        qkv = normal(b, lq, h + 2 * hk, d)
        s["q"], s["k"], s["v"] = qkv[:, :, :h], qkv[:, :, h:h + hk], qkv[:, :, h + hk:]
    else:
        kv = normal(b, lk, 2 * hk, d)
        s["q"], s["k"], s["v"] = normal(b, lq, h, d), kv[:, :, :hk], kv[:, :, hk:]
    s["lens"] = None
    if case["fill"] < 1.0:
        order = torch.randperm(b, device=DEV, generator=g)
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)[order].contiguous()
    s["bias"], s["borders"] = None, None
    if case["buckets"]:
        s["borders"] = _borders(case["buckets"], case["far"], s["two_sided"])
        s["bias"] = torch.randn(case["buckets"], h, device=DEV, generator=g)
    if case["op"] == "attn_bwd":
        s["dout"] = normal(b, lq, h, d, std=0.02)
        out, lse = _plain_forward(s)
        s["out"], s["lse"] = out, lse
    return s


def _layer_input(rows, d, dtype, g):
    """Rectified activations, a tenth of the columns a hundred times larger."""
    x = torch.randn(rows, d, device=DEV, generator=g).clamp_min_(0)
    x[:, torch.rand(d, device=DEV, generator=g) < 0.1] *= 100.0
    return x.to(dtype)


def prepare(case, seed):
    if case["op"].startswith("attn"):
        return _attn_state(case, seed)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rows, d = case["rows"], case["d"]
    s = {"case": case, "rows": rows}
    x = _layer_input(rows, d, _type(case), g)
    if case["op"] == "keep":
        s["x"] = x
        return s
    s["codes"], s["scales"] = _plain_store(x, case["ones"])
    da = d + int(case["ones"])
    if case["op"] == "factor":
        s["m"] = torch.zeros(da, da, device=DEV)
    else:
        s["g"] = (torch.randn(rows, case["d_out"], device=DEV, generator=g) * 1e-3).to(_type(case))
    return s


# ------------------------------------------------------------- plain forms --

def _bucket_of(s):
    """Bucket of every offset key - query, from -(len_q - 1) to len_k - 1 places from the first query's."""
    c = s["case"]
    lq, lk = c["len_q"], c["len_k"]
    rel = torch.arange(lq + lk - 1, device=DEV) - (lq - 1) - (lk - lq)
    edges = torch.tensor(s["borders"], device=DEV)
    if not s["two_sided"]:
        return torch.searchsorted(edges, (-rel).clamp_min(0), right=True)
    return torch.searchsorted(edges, rel.abs(), right=True) + (rel > 0) * (len(s["borders"]) + 1)


def _hidden(s):
    """[batch, 1, len_q, len_k]: key not visible to query."""
    c = s["case"]
    lq, lk = c["len_q"], c["len_k"]
    j = torch.arange(lk, device=DEV)
    hid = torch.zeros(1, 1, lq, lk, dtype=torch.bool, device=DEV)
    if c["causal"]:
        hid = hid | (j > (torch.arange(lq, device=DEV) + (lk - lq))[:, None])
    if s["lens"] is not None:
        hid = hid | (j >= s["lens"][:, None, None, None])
    return hid


def _heads_first(x, repeat=1):
    x = x.float().transpose(1, 2)
    return x.repeat_interleave(repeat, dim=1) if repeat > 1 else x.contiguous()


def _scores(s):
    c = s["case"]
    lq, lk = c["len_q"], c["len_k"]
    r = c["heads"] // c["kv_heads"]
    w = torch.matmul(_heads_first(s["q"]) * s["scale"], _heads_first(s["k"], r).transpose(2, 3).contiguous())
    if s["bias"] is not None:
        at = torch.arange(lk, device=DEV) - torch.arange(lq, device=DEV)[:, None] + (lq - 1)
        w += s["bias"].t()[:, _bucket_of(s)][:, at]
    return w.masked_fill_(_hidden(s), -math.inf)


def _plain_forward(s):
    w = _scores(s)
    top = w.amax(dim=3, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(w.sub_(top))
    total = w.sum(dim=3, keepdim=True)
    r = s["case"]["heads"] // s["case"]["kv_heads"]
    out = torch.matmul(w, _heads_first(s["v"], r)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).squeeze(3)
    return out.transpose(1, 2).contiguous().to(s["q"].dtype), lse


def _plain_backward(s):
    c, t = s["case"], s["q"].dtype
    b, lq, lk, h, hk, d = (c[k] for k in ("batch", "len_q", "len_k", "heads", "kv_heads", "dim"))
    r = h // hk
    lse = s["lse"].unsqueeze(3)
    p = torch.exp(_scores(s).sub_(torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)))
    do, v = _heads_first(s["dout"]), _heads_first(s["v"], r)
    delta = (do * _heads_first(s["out"])).sum(dim=3, keepdim=True)

    def back(x, groups):
        x = x.reshape(b, groups, -1, x.shape[2], d).sum(dim=2)
        return x.transpose(1, 2).contiguous().to(t)

    dv = back(torch.matmul(p.transpose(2, 3).contiguous(), do), hk)
    ds = torch.matmul(do, v.transpose(2, 3).contiguous()).sub_(delta).mul_(p)
    del p
    dq = back(torch.matmul(ds, _heads_first(s["k"], r)) * s["scale"], h)
    dk = back(torch.matmul(ds.transpose(2, 3).contiguous(), _heads_first(s["q"])) * s["scale"], hk)
    got = {"dq": dq, "dk": dk, "dv": dv}
    if s["bias"] is not None:
        # rows turned over and laid one element further each: the columns then hold one offset each
        flat = torch.nn.functional.pad(ds.sum(dim=0).flip(1), (0, lq)).reshape(h, lq * (lq + lk))
        width = lq + lk - 1
        along = flat[:, :lq * width].reshape(h, lq, width).sum(dim=1, dtype=torch.float64)
        table = torch.zeros(c["buckets"], h, dtype=torch.float64, device=DEV)
        got["dbias"] = table.index_add_(0, _bucket_of(s), along.t().contiguous()).float()
    return got


def _power(e):
    """2^e in float32 from its bits, e in [-126, 127] (pow and exp2 on a GPU may miss a power of two by a rounding)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_store(x, ones):
    rows = x.shape[0]
    x = x.float()
    if ones:
        x = torch.cat([x, torch.ones(rows, 1, device=DEV)], dim=1)
    blocks = (rows + 31) // 32
    x = torch.nn.functional.pad(x, (0, 0, 0, blocks * 32 - rows)).reshape(blocks, 32, -1)
    top = x.abs().amax(dim=1)
    part, e = torch.frexp(top)                            # top = part 2^e, part in [0.5, 1)
    e = torch.where(part > 0.875, e - 8, e - 9).clamp_min(MIN_EXP)   # 448 = 0.875 2^9
    e = torch.where(top > 0, e, torch.full_like(e, MIN_EXP))
    codes = (x.double() * _power(-e.unsqueeze(1)).double()).float().to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).transpose(1, 2).contiguous(), (e + 127).to(torch.uint8)


def _plain_load(codes, scales, rows):
    x = codes.view(torch.float8_e4m3fn).float() * _power(scales.to(torch.int32) - 127).unsqueeze(2)
    return x.transpose(1, 2).reshape(-1, codes.shape[1])[:rows]


# ------------------------------------------------------------------ one pass --

def _own_attention(s):
    import linear_algebra_amd as la

    c = s["case"]
    b, lq, h = c["batch"], c["len_q"], c["heads"]
    form = dict(scale=s["scale"], causal=c["causal"], lens=s["lens"], bias=s["bias"], borders=s["borders"],
                two_sided=s["two_sided"])
    if c["op"] == "attn_fwd":
        out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
        lse = torch.empty(b, h, lq, device=DEV)
        la.kfac_attention_forward(s["q"], s["k"], s["v"], out, lse, **form)
        return {"out": out, "lse": lse}
    got = {"d" + n: torch.empty(s[n].shape, dtype=s[n].dtype, device=DEV) for n in ("q", "k", "v")}
    if s["bias"] is not None:
        got["dbias"] = torch.empty_like(s["bias"])
    la.kfac_attention_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], got["dq"], got["dk"], got["dv"],
                               dbias=got.get("dbias"), **form)
    return got


def _own_checkpoint(s):
    import linear_algebra_amd as la

    c, rows = s["case"], s["rows"]
    if c["op"] == "keep":
        da = c["d"] + int(c["ones"])
        codes, scales = la.kfac_checkpoint_empty(rows, da, DEV)
        la.kfac_checkpoint_store([s["x"]], [codes], [scales], ones=c["ones"])
        values = torch.empty(rows, da, dtype=s["x"].dtype, device=DEV)
        la.kfac_checkpoint_load([codes], [scales], [values])
        return {"scales": scales, "values": values}
    if c["op"] == "factor":
        la.kfac_checkpoint_factors([s["codes"]], [s["scales"]], [rows], [s["m"]], 0.95, True)
        return {"m": s["m"]}
    mat = torch.empty(c["d_out"], s["codes"].shape[1], device=DEV)
    la.kfac_checkpoint_grad([s["g"]], [s["codes"]], [s["scales"]], [mat])
    return {"mat": mat}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _own_attention(s) if op.startswith("attn") else _own_checkpoint(s)
    if op == "attn_fwd":
        out, lse = _plain_forward(s)
        return {"out": out, "lse": lse}
    if op == "attn_bwd":
        return _plain_backward(s)
    if op == "keep":
        codes, scales = _plain_store(s["x"], s["case"]["ones"])
        return {"scales": scales, "values": _plain_load(codes, scales, s["rows"]).to(s["x"].dtype)}
    x = _plain_load(s["codes"], s["scales"], s["rows"])
    if op == "factor":
        # the upper triangle is the factor; below it the caller's buffer keeps its zeros
        return {"m": s["m"].copy_(torch.triu(torch.matmul(x.t(), x) / s["rows"]))}
    return {"mat": torch.matmul(s["g"].float().t(), x)}


# ------------------------------------------------------------------- 64 bits --

def _exact_visible(s, b):
    c = s["case"]
    i = torch.arange(c["len_q"], device=DEV).reshape(-1, 1) + c["len_k"] - c["len_q"]
    j = torch.arange(c["len_k"], device=DEV).reshape(1, -1)
    see = (j <= i) if c["causal"] else (j > -1).expand(c["len_q"], c["len_k"])
    if s["lens"] is not None:
        see = see & (j < int(s["lens"][b]))
    bucket = None
    if s["bias"] is not None:
        gap = (i - j).abs() if s["two_sided"] else (i - j).clamp_min(0)
        bucket = torch.zeros(c["len_q"], c["len_k"], dtype=torch.int64, device=DEV)
        for edge in s["borders"]:
            bucket += gap >= edge
        if s["two_sided"]:
            bucket += (j > i) * (len(s["borders"]) + 1)
    return see, bucket


def _exact_attention(s):
    """Head by head, in float64: the probabilities as exp(score) over their sum (forward), as exp(score - lse) (backward)."""
    c = s["case"]
    f64 = dict(dtype=torch.float64, device=DEV)
    group = c["heads"] // c["kv_heads"]
    if c["op"] == "attn_fwd":
        got = {"out": torch.zeros(s["q"].shape, **f64),
               "lse": torch.full((c["batch"], c["heads"], c["len_q"]), -math.inf, **f64)}
    else:
        got = {"d" + n: torch.zeros(s[n].shape, **f64) for n in ("q", "k", "v")}
        if s["bias"] is not None:
            got["dbias"] = torch.zeros(s["bias"].shape, **f64)
    for b in range(c["batch"]):
        see, bucket = _exact_visible(s, b)
        some = see.any(dim=1)
        for h in range(c["heads"]):
            kv = h // group
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :, kv].double(), s["v"][b, :, kv].double()
            score = q @ k.t() * s["scale"]
            if bucket is not None:
                score = score + s["bias"][:, h].double()[bucket]
            if c["op"] == "attn_fwd":
                top = torch.where(see, score, torch.full_like(score, -math.inf)).amax(dim=1).nan_to_num(neginf=0.0)
                e = torch.exp(score - top[:, None]) * see
                z = e.sum(dim=1)
                got["lse"][b, h] = torch.log(z) + top
                got["out"][b, :, h] = (e / torch.where(some, z, torch.ones_like(z))[:, None]) @ v
                continue
            lse = s["lse"][b, h].double()
            p = torch.exp(score - torch.where(some, lse, torch.zeros_like(lse))[:, None])
            p = torch.where(see, p, torch.zeros_like(p))
            do = s["dout"][b, :, h].double()
            delta = (do * s["out"][b, :, h].double()).sum(dim=1)
            ds = p * (do @ v.t() - delta[:, None])
            got["dq"][b, :, h] = ds @ k * s["scale"]
            got["dk"][b, :, kv] += ds.t() @ q * s["scale"]
            got["dv"][b, :, kv] += p.t() @ do
            if bucket is not None:
                for n in range(s["bias"].shape[0]):
                    got["dbias"][n, h] += (ds * (bucket == n)).sum()
    return got


def _scaled(x, e):
    """x 2^e in float64, the power from its bits."""
    return x * ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(codes, scales, rows):
    """sign (1 + m / 8) 2^(e - 7), or m / 8 2^-6 where e is 0, times the block's power of two."""
    n = codes.to(torch.int64)
    sign, e, m = 1 - 2 * (n >> 7), (n >> 3) & 15, (n & 7).double()
    x = torch.where(e == 0, m / 8 / 64, _scaled(1 + m / 8, e - 7)) * sign
    x = _scaled(x, scales.to(torch.int64)[:, :, None] - 127)
    return x.permute(0, 2, 1).reshape(-1, codes.shape[1])[:rows]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("attn"):
        return _exact_attention(s)
    rows = case["rows"]
    if case["op"] == "keep":
        x = s["x"].double()
        if case["ones"]:
            x = torch.cat([x, torch.ones_like(x[:, :1])], dim=1)
        blocks = -(-rows // 32)
        full = torch.zeros(blocks * 32, x.shape[1], dtype=torch.float64, device=DEV)
        full[:rows] = x
        full = full.reshape(blocks, 32, -1)
        top = full.abs().amax(dim=1)
        e = torch.full_like(top, MIN_EXP, dtype=torch.int64)
        for n in range(MIN_EXP, 121):
            e[top > E4M3_MAX * 2.0 ** n] = n + 1
        y = _scaled(full, -e[:, None])
        step = _scaled(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp_min(-6) - 3)
        y = _scaled(torch.round(y / step) * step, e[:, None])
        return {"scales": (e + 127).to(torch.uint8), "values": y.reshape(blocks * 32, -1)[:rows]}
    x = _exact_values(s["codes"], s["scales"], rows)
    if case["op"] == "factor":
        return {"m": torch.triu(x.t() @ x / rows)}
    return {"mat": s["g"].double().t() @ x}
