"""GPU: attention with a bucketed relative position bias, forward and
backward, against the float64 form, within bounds derived from the roundings."""
import pytest

import linear_algebra_amd as la
from tests import training_reference as ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

BORDERS = [1, 2, 3, 4, 6, 9, 14, 22, 40]
# dtype, batch, len_q, len_k, heads, kv_heads, dim, causal, two_sided, borders (None: no bias), lens
CASES = [
    ("bf16", 1, 1, 1, 1, 1, 8, False, True, None, None),
    ("f32", 1, 1, 1, 1, 1, 8, True, True, [], None),
    ("bf16", 2, 1, 77, 3, 1, 40, False, True, BORDERS, [77, 1]),
    ("bf16", 1, 77, 1, 2, 2, 32, False, True, BORDERS, None),
    ("bf16", 2, 31, 33, 2, 2, 16, False, False, [1, 5], None),
    ("bf16", 2, 64, 64, 4, 2, 64, True, True, BORDERS, None),
    ("bf16", 1, 127, 127, 2, 1, 72, True, False, BORDERS, None),
    ("bf16", 1, 128, 128, 2, 2, 96, False, True, BORDERS, None),
    ("bf16", 3, 129, 200, 3, 1, 128, False, True, BORDERS, [0, 65, 200]),
    ("bf16", 2, 300, 300, 6, 2, 128, True, True, list(range(1, 64)), [300, 170]),
    ("bf16", 2, 300, 257, 2, 2, 64, True, False, BORDERS, None),       # queries before every key: empty rows
    ("bf16", 1, 130, 400, 2, 1, 64, True, True, BORDERS, [399]),
    ("bf16", 1, 1100, 1100, 2, 1, 64, True, False, BORDERS, None),
    ("bf16", 1, 260, 260, 2, 1, 64, False, True, [200], None),
    ("f32", 2, 33, 65, 4, 2, 24, False, True, BORDERS, [65, 0]),
    ("f32", 1, 200, 200, 2, 1, 64, True, True, BORDERS, None),
    ("f32", 2, 129, 129, 3, 3, 96, False, False, BORDERS, [129, 31]),
    ("f32", 1, 257, 257, 2, 1, 128, True, False, list(range(1, 128)), None),
    ("f32", 1, 140, 300, 2, 2, 128, False, True, None, [290]),
    ("bf16", 2, 150, 150, 2, 1, 64, True, True, [1, 7, 30, 5000], None),   # a stretch too long for the LDS table
    ("f32", 1, 70, 90, 2, 2, 32, False, False, [3, 2000], None),
    ("bf16", 1, 2500, 600, 2, 2, 32, False, True, [1, 2, 8, 1500], None),
]


def make(case, seed=0, layout="plain"):
    import torch
    dtype, b, lq, lk, h, hk, d, causal, two_sided, borders, lens = case
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(seed)
    s = {"case": case, "q": torch.randn(b, lq, h, d, generator=g).to(t), "k": torch.randn(b, lk, hk, d, generator=g).to(t),
         "v": torch.randn(b, lk, hk, d, generator=g).to(t), "dout": torch.randn(b, lq, h, d, generator=g).to(t)}
    s["form"] = dict(scale=d ** -0.5, causal=causal, two_sided=two_sided, lens=None, bias=None, borders=borders or [])
    if lens is not None:
        s["form"]["lens"] = torch.tensor(lens, dtype=torch.int32)
    if borders is not None:
        n = (len(borders) + 1) * (2 if two_sided else 1)
        s["form"]["bias"] = torch.randn(n, h, generator=g)
    return s


def on_dev(t, layout):
    """The tensor on the GPU: rows first, heads first, or as part of a wider row."""
    import torch
    if layout == "heads":
        return t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    if layout == "part":
        wide = torch.full((t.shape[0], t.shape[1], t.shape[2] + 2, t.shape[3]), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, :, 1:-1] = t.to(DEV)
        return wide[:, :, 1:-1]
    return t.to(DEV)


def dev_form(form):
    f = dict(form)
    for n in ("lens", "bias"):
        if f[n] is not None:
            f[n] = f[n].to(DEV)
    if f["bias"] is None:
        f["borders"] = None
    return f


def new(like, layout):
    import torch
    return on_dev(torch.full(like.shape, float("nan"), dtype=like.dtype), layout)


def forward(s, layout="plain", stream=None):
    import torch
    q, k, v = (on_dev(s[n], layout) for n in "qkv")
    out = new(s["q"], layout)
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), float("nan"), device=DEV)
    f = dev_form(s["form"])
    torch.cuda.synchronize()
    la.kfac_attention_forward(q, k, v, out, lse, stream=stream, **f)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def backward(s, out, lse, layout="plain", stream=None):
    import torch
    q, k, v, do, o = (on_dev(t, layout) for t in (s["q"], s["k"], s["v"], s["dout"], out))
    got = {"d" + n: new(s[n], layout) for n in "qkv"}
    f = dev_form(s["form"])
    got["dbias"] = torch.full_like(f["bias"], float("nan")) if f["bias"] is not None else None
    lse = lse.to(DEV)
    torch.cuda.synchronize()
    la.kfac_attention_backward(q, k, v, o, lse, do, got["dq"], got["dk"], got["dv"], got["dbias"], stream=stream, **f)
    torch.cuda.synchronize()
    return {n: t.cpu() for n, t in got.items() if t is not None}


def check(name, got, want, bound):
    import torch
    got = got.double()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf), name
    err = (got - want).abs()[~inf]
    assert not torch.isnan(err).any(), name
    lim = bound[~inf]
    worst = float((err / lim.clamp_min(1e-300)).max()) if err.numel() else 0.0
    say(f"  {name}: error at most {worst:.3f} of its bound")
    assert bool((err <= lim).all()), (name, worst)


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-{c[0]}-{c[2]}x{c[3]}x{c[6]}" for i, c in enumerate(CASES)])
def test_attention(case):
    s = make(case)
    say("attention", case)
    layout = ("plain", "heads", "part")[CASES.index(case) % 3]
    out, lse = forward(s, layout)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], **s["form"])
    for n, t in (("out", out), ("lse", lse)):
        check(n, t, *want[n])
    got = backward(s, out, lse, layout)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], out=out, lse=lse, dout=s["dout"], **s["form"])
    assert set(got) == set(want)
    for n in want:
        check(n, got[n], *want[n])


MANY_HEADS = [   # sequences times heads of keys: multiples of eight, few more than eight, and odd ones
    ("bf16", 4, 130, 40, 8, 8, 32, False, True, BORDERS, [0, 40, 7, 33]),
    ("bf16", 6, 33, 300, 12, 6, 64, False, True, BORDERS, [300, 0, 129, 1, 256, 128]),
    ("bf16", 40, 260, 40, 16, 8, 16, True, False, BORDERS, None),
    ("f32", 17, 40, 20, 2, 1, 16, False, True, BORDERS, None),
    ("f32", 3, 64, 64, 9, 9, 8, True, False, BORDERS, [64, 3, 0]),
    ("bf16", 24, 300, 257, 8, 8, 24, False, True, None, list(range(3, 243, 10))),
]


@pytest.mark.parametrize("case", MANY_HEADS, ids=[f"{c[1]}x{c[4]}" for c in MANY_HEADS])
def test_sequences_and_heads_dealt_out(case):
    """Every sequence and head is computed once, whatever their number."""
    s = make(case, 7)
    say("many heads", case)
    out, lse = forward(s)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], **s["form"])
    for n, t in (("out", out), ("lse", lse)):
        check(n, t, *want[n])
    got = backward(s, out, lse)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], out=out, lse=lse, dout=s["dout"], **s["form"])
    assert set(got) == set(want)
    for n in want:
        check(n, got[n], *want[n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_hidden_keys_hold_anything(dtype):
    """NaN and infinities past a sequence's length change nothing, and their gradients are 0."""
    import torch
    case = (dtype, 3, 70, 150, 2, 1, 64, False, True, BORDERS, [0, 97, 150])
    s = make(case)
    out, lse = forward(s)
    got = backward(s, out, lse)
    for b, n in enumerate(case[-1]):
        s["k"][b, n:] = float("nan")
        s["v"][b, n:] = float("inf")
    out2, lse2 = forward(s)
    got2 = backward(s, out, lse)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for n in got:
        assert torch.equal(got[n], got2[n]), n
    for b, n in enumerate(case[-1]):
        assert not got["dk"][b, n:].any() and not got["dv"][b, n:].any()
    assert not out[0].any() and bool((lse[0] == -float("inf")).all()) and not got["dq"][0].any()


def test_empty_lengths():
    import torch
    for lq, lk in ((0, 5), (5, 0), (0, 0)):
        say("lengths", lq, lk)
        s = make(("bf16", 2, lq, lk, 2, 1, 16, False, True, [1, 4], None))
        out, lse = forward(s)
        assert not out.any() and bool((lse == -float("inf")).all())
        got = backward(s, out, lse)
        assert all(not t.any() for t in got.values())


def test_broadcast_keys():
    """Keys and values expanded along the batch (stride 0): gradients come back per sequence."""
    import torch
    s = make(("bf16", 3, 65, 90, 2, 2, 32, False, True, BORDERS, None))
    s["k"], s["v"] = s["k"][:1].expand(3, -1, -1, -1), s["v"][:1].expand(3, -1, -1, -1)
    k, v = s["k"][:1].contiguous().to(DEV).expand(3, -1, -1, -1), s["v"][:1].contiguous().to(DEV).expand(3, -1, -1, -1)
    out, lse = forward(s)
    o2, l2 = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV), torch.empty(lse.shape, device=DEV)
    la.kfac_attention_forward(s["q"].to(DEV), k, v, o2, l2, **dev_form(s["form"]))
    assert torch.equal(o2.cpu(), out) and torch.equal(l2.cpu(), lse)


def test_same_bits_every_run_and_on_another_stream():
    import torch
    for case in (CASES[9], CASES[8], CASES[15]):
        s = make(case, 5)
        out, lse = forward(s)
        got = backward(s, out, lse)
        side = torch.cuda.Stream()
        out2, lse2 = forward(s, stream=side)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        for _ in range(2):
            again = backward(s, out, lse, stream=side)
            for n in got:
                assert torch.equal(got[n], again[n]), n


def test_captured_in_a_graph():
    import torch
    s = make(CASES[9], 6)
    q, k, v, do = (s[n].to(DEV) for n in ("q", "k", "v", "dout"))
    f = dev_form(s["form"])

    def step(r):
        la.kfac_attention_forward(q, k, v, r["out"], r["lse"], **f)
        la.kfac_attention_backward(q, k, v, r["out"], r["lse"], do, r["dq"], r["dk"], r["dv"], r["dbias"], **f)

    def room():
        return {"out": torch.zeros_like(q), "lse": torch.zeros(q.shape[0], q.shape[2], q.shape[1], device=DEV),
                "dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v),
                "dbias": torch.zeros_like(f["bias"])}

    cap, eager = room(), room()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for replay in range(3):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(replay)).to(q.dtype))
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for n in cap:
            assert torch.equal(cap[n], eager[n]), (replay, n)


def test_forward_differences():
    """The gradients against differences of the kernel's own forward pass, in
    float32.  With r = sum(out w), the difference over 2 h along a unit
    direction is off by h^2 / 6 times the third derivative (below 50 here: the
    softmax's, for scores with slopes of order one) and by the forward's
    rounding, 2^-24 times a few hundred terms of order one, over h."""
    import torch
    s = make(("f32", 1, 48, 48, 2, 1, 32, True, True, BORDERS, None), 7)
    w = s["dout"].double()
    out, lse = forward(s)
    got = backward(s, out, lse)
    h = 2e-2
    for name in ("q", "k", "v", "bias"):
        x = s["form"]["bias"] if name == "bias" else s[name]
        d = torch.randn(x.shape, generator=torch.Generator().manual_seed(8))
        d = d / d.norm()
        r = []
        for sign in (1, -1):
            t = dict(s)
            if name == "bias":
                t["form"] = dict(s["form"], bias=x + sign * h * d)
            else:
                t[name] = x + sign * h * d
            r.append(float((forward(t)[0].double() * w).sum()))
        diff = (r[0] - r[1]) / (2 * h)
        formula = float((got["dbias" if name == "bias" else "d" + name].double() * d.double()).sum())
        say(f"  {name}: formula {formula:.6f}, difference {diff:.6f}")
        assert abs(diff - formula) <= 50 * h * h / 6 + 4096 * 2.0 ** -24 * 4 / h


def test_many_bias_sums():
    """More pairs of head and bucket than key tiles by far: every entry of the bias gradient is written."""
    case = ("bf16", 1, 4, 5, 4096, 512, 8, False, True, list(range(1, 64)), None)
    s = make(case, 9)
    say("many sums", case)
    out, lse = forward(s)
    got = backward(s, out, lse)
    want = ref.attention(s["q"], s["k"], s["v"], dtype="bf16", out=out, lse=lse, dout=s["dout"], **s["form"])
    for n in want:
        check(n, got[n], *want[n])


LONG_BORDERS = [   # stretches too long for the LDS table, where the last step of a chunk has no queries left
    ("f32", 1, 128, 128, 4, 4, 64, False, True, [1, 7, 30, 2048], None),
    ("f32", 2, 128, 128, 4, 2, 72, True, False, [2, 2000], [128, 50]),
    ("bf16", 1, 1024, 1024, 5, 5, 64, False, True, [3, 40, 1200], None),
    ("bf16", 2, 384, 384, 16, 16, 64, False, True, [1, 1000], None),
    ("bf16", 8, 127, 1, 5, 5, 32, True, True, [1, 1200], None),
]


@pytest.mark.parametrize("case", LONG_BORDERS, ids=[f"{c[0]}-{c[1]}x{c[2]}x{c[6]}" for c in LONG_BORDERS])
def test_bias_is_read_inside_the_workspace(case, monkeypatch):
    """The bytes in front of and behind the workspace are NaN, and none of them reaches a gradient."""
    import torch

    def fenced(need, device, name):
        ws = torch.full((need + 8192,), 0xFF, dtype=torch.uint8, device=device)
        return ws, ws.data_ptr() + 4096, need

    s = make(case, 3)
    say("long borders", case)
    out, lse = forward(s)
    monkeypatch.setattr(la, "_space", fenced)
    got = backward(s, out, lse)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], out=out, lse=lse, dout=s["dout"], **s["form"])
    assert set(got) == set(want)
    for n in want:
        check(n, got[n], *want[n])


ABSENT = [   # an odd count of query steps, a last step of which half is missing, shared and unshared key tiles
    ("bf16", 1, 77, 77, 2, 1, 64, False, True, BORDERS, None),
    ("bf16", 1, 33, 50, 2, 2, 32, False, True, BORDERS, [44]),
    ("bf16", 2, 20, 20, 4, 2, 128, True, False, BORDERS, None),
    ("bf16", 40, 65, 40, 16, 16, 16, True, True, BORDERS, None),
    ("f32", 1, 32, 32, 2, 2, 64, False, True, BORDERS, None),
    ("f32", 2, 70, 90, 3, 1, 72, True, True, BORDERS, [90, 41]),
]


@pytest.mark.parametrize("case", ABSENT, ids=[f"{c[0]}-{c[1]}x{c[2]}x{c[6]}" for c in ABSENT])
def test_large_biases(case):
    """A common offset of the bias, past the largest exponential of float32,
    changes the logarithms and nothing else: places past the last query, whose
    numbers it would make infinite, add nothing.  The sums of a score begin
    with a number of the offset's size: up to dim roundings more at its size."""
    import torch
    s = make(case, 11)
    s["form"]["bias"] += 100.0
    say("large biases", case)
    out, lse = forward(s)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], **s["form"])
    for n, t in (("out", out), ("lse", lse)):
        check(n, t, *want[n])
    got = backward(s, out, lse)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], out=out, lse=lse, dout=s["dout"], roundings=16 + case[6],
                         **s["form"])
    assert set(got) == set(want)
    for n in want:
        check(n, got[n], *want[n])


REPEATED = [("bf16", 1, 77, 77, 2, 1, 64, False, True, BORDERS, None), ("bf16", 2, 1, 40, 2, 2, 32, False, True, None, None),
            ("bf16", 1, 130, 130, 2, 2, 128, True, True, BORDERS, None), ("f32", 2, 33, 50, 2, 1, 64, False, False, BORDERS, [50, 9]),
            ("bf16", 40, 65, 40, 16, 16, 16, False, True, None, None)]


@pytest.mark.parametrize("case", REPEATED, ids=[f"{c[0]}-{c[2]}x{c[3]}x{c[6]}" for c in REPEATED])
@pytest.mark.parametrize("which", ["dout", "q", "kv"])
def test_repeated_rows(case, which):
    """One row for every query or key (row stride 0), as a sum over the rows sends back: the same bits as its copies."""
    import torch
    s = make(case, 12)
    names = {"dout": ["dout"], "q": ["q"], "kv": ["k", "v"]}[which]
    for n in names:
        s[n] = s[n][:, :1].expand(s[n].shape).contiguous()
    say("repeated rows", which, case)
    out, lse = forward(s)
    want = backward(s, out, lse)
    dev = {n: s[n].to(DEV) for n in ("q", "k", "v", "dout")}
    for n in names:
        dev[n] = dev[n][:, :1].expand(s[n].shape)
        assert dev[n].stride(1) == 0 or dev[n].shape[1] == 1
    f = dev_form(s["form"])
    o, l = torch.empty_like(out, device=DEV), torch.empty_like(lse, device=DEV)
    la.kfac_attention_forward(dev["q"], dev["k"], dev["v"], o, l, **f)
    assert torch.equal(o.cpu(), out) and torch.equal(l.cpu(), lse)
    got = {"d" + n: torch.full(s[n].shape, float("nan"), dtype=s[n].dtype, device=DEV) for n in "qkv"}
    if f["bias"] is not None:
        got["dbias"] = torch.full_like(f["bias"], float("nan"))
    la.kfac_attention_backward(dev["q"], dev["k"], dev["v"], o, l, dev["dout"], got["dq"], got["dk"], got["dv"],
                               got.get("dbias"), **f)
    for n in want:
        assert torch.equal(got[n].cpu(), want[n]), n


# Passes by queries with 192 workgroups of 128 queries and more, which take 128
# queries per workgroup (tests/test_training_host.py holds every case to that),
# at each head width that has kernels of its own.
WIDE = [
    ("bf16", 4, 130, 200, 24, 8, 32, False, True, BORDERS, [200, 0, 77, 129]),
    ("bf16", 8, 300, 300, 8, 8, 64, True, True, BORDERS, None),
    ("bf16", 4, 140, 200, 24, 8, 64, False, True, BORDERS, [0, 200, 64, 65]),
    ("bf16", 4, 140, 140, 24, 12, 96, True, False, [1, 2, 5, 30, 60], [140, 1, 99, 140]),
    ("bf16", 6, 257, 130, 16, 4, 128, False, False, BORDERS, [130, 0, 64, 33, 96, 1]),
    ("bf16", 3, 200, 333, 32, 8, 128, True, True, None, None),
    ("bf16", 2, 300, 260, 32, 8, 72, True, True, BORDERS, [260, 100]),           # queries before every key
    ("bf16", 4, 150, 150, 24, 24, 64, False, True, [1, 7, 30, 5000], None),      # a stretch too long for the LDS table
    ("bf16", 4, 150, 180, 24, 12, 128, True, False, [1, 2000], [180, 9, 0, 64]),
    ("f32", 4, 130, 90, 24, 8, 32, False, True, BORDERS, [90, 0, 33, 64]),
    ("f32", 8, 300, 300, 8, 4, 64, True, True, BORDERS, None),
    ("f32", 4, 200, 257, 24, 12, 72, False, False, BORDERS, [257, 31, 0, 128]),
    ("f32", 4, 140, 140, 24, 24, 96, False, True, None, [140, 7, 33, 96]),
    ("f32", 4, 129, 140, 24, 8, 128, True, False, BORDERS, None),
    ("f32", 4, 150, 150, 24, 12, 64, False, True, [1, 7, 30, 2000], None),
]
# ... and with 512 key tiles and more, which are not shared out.
UNSHARED = [
    ("bf16", 64, 40, 40, 8, 8, 64, True, True, BORDERS, None),
    ("bf16", 32, 77, 140, 16, 8, 128, False, True, BORDERS, [5 * n % 141 for n in range(32)]),
    ("bf16", 32, 33, 300, 12, 6, 96, True, False, BORDERS, None),
    ("bf16", 40, 70, 90, 16, 16, 64, False, True, None, [7 * n % 91 for n in range(40)]),
    ("bf16", 32, 70, 150, 8, 8, 128, False, True, [1, 1500], None),
    ("f32", 32, 33, 300, 6, 6, 128, False, True, BORDERS, [300 - 9 * n for n in range(32)]),
    ("f32", 64, 40, 40, 16, 8, 64, True, True, BORDERS, None),
    ("f32", 64, 50, 30, 8, 8, 72, False, False, None, None),
    ("f32", 64, 20, 40, 8, 8, 32, False, True, [2, 2000], None),
]


@pytest.mark.parametrize("case", WIDE + UNSHARED, ids=[f"{i}-{c[0]}-{c[1]}x{c[2]}x{c[3]}x{c[6]}" for i, c in enumerate(WIDE + UNSHARED)])
def test_many_queries(case):
    s = make(case, 13)
    say("many queries", case)
    layout = ("plain", "heads", "part")[(WIDE + UNSHARED).index(case) % 3]
    out, lse = forward(s, layout)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], **s["form"])
    for n, t in (("out", out), ("lse", lse)):
        check(n, t, *want[n])
    got = backward(s, out, lse, layout)
    want = ref.attention(s["q"], s["k"], s["v"], dtype=case[0], out=out, lse=lse, dout=s["dout"], **s["form"])
    assert set(got) == set(want)
    for n in want:
        check(n, got[n], *want[n])
