"""GPU: the gated feed-forward block forward and backward against float64
forms, elementwise within what the formulas' roundings allow."""
import pytest

import linear_algebra_amd as la
from tests import encoder_reference as ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

ACTS = list(la.KFAC_ACTIVATIONS)
# rows, d, width: one of each, less than a block, both sides of blocks and
# tiles, odd widths, long and short reductions
SHAPES = [(1, 1, 1), (1, 8, 2), (2, 3, 5), (1, 64, 64), (3, 16, 7), (15, 40, 16), (16, 513, 100), (17, 130, 97), (31, 33, 32),
          (32, 64, 33), (33, 65, 63), (64, 70, 64), (65, 100, 65), (127, 129, 127), (128, 128, 128), (129, 127, 129),
          (130, 250, 66), (200, 8, 300), (257, 640, 70), (5, 1000, 300), (300, 72, 1), (1, 2048, 512), (70, 2, 260),
          (513, 34, 21), (1100, 260, 390)]


def inputs(rows, d, width, dtype, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed + 31 * rows + 7 * d + width)
    t = ref.types()[dtype]

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    return (normal(rows, d).to(t), (normal(2 * width, d) * d ** -0.5).to(t), normal(2 * width), (normal(rows, 2 * width) * 2).to(t),
            normal(rows, width).to(t))


def nan(*shape, dtype):
    import torch
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def forward(x, w, b, act, keep=True):
    rows, width = x.shape[0], w.shape[0] // 2
    h = nan(rows, width, dtype=x.dtype)
    pre = nan(rows, 2 * width, dtype=x.dtype) if keep else None
    la.kfac_gated_forward(x.to(DEV), w.to(DEV), h, bias=None if b is None else b.to(DEV), pre=pre, activation=act)
    return h, pre


def backward(dh, x, w, pre, act, dweight_type=None):
    import torch
    rows, d, width = x.shape[0], x.shape[1], w.shape[0] // 2
    got = {"dpre": nan(rows, 2 * width, dtype=x.dtype), "dx": nan(rows, d, dtype=x.dtype),
           "dweight": nan(2 * width, d, dtype=dweight_type or x.dtype), "dbias": nan(2 * width, dtype=torch.float32)}
    la.kfac_gated_backward(*(t.to(DEV) for t in (dh, x, w, pre)), activation=act, **got)
    return got


def hold(got, want):
    for name in want:
        if got.get(name) is not None:
            r = ref.worst(got[name], *want[name])
            say(f"  {name} {r:.3f}")
            assert r <= 1.0, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,width", SHAPES)
def test_forward(rows, d, width, dtype):
    act = ACTS[(rows + d) % len(ACTS)]
    x, w, b, _, _ = inputs(rows, d, width, dtype)
    h, pre = forward(x, w, b, act)
    hold({"h": h, "pre": pre}, ref.gated_forward(x, w, b, act, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,width", SHAPES)
def test_backward(rows, d, width, dtype):
    act = ACTS[(rows + d + 2) % len(ACTS)]
    x, w, b, pre, dh = inputs(rows, d, width, dtype)
    got = backward(dh, x, w, pre, act)
    hold(got, ref.gated_backward(dh, x, w, pre, got["dpre"].cpu(), act, dtype, dtype))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activations(dtype, act):
    """Values from the smallest to where the activation saturates, and past it."""
    import torch
    t = ref.types()[dtype]
    gate = torch.cat([torch.linspace(-12, 12, 97), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 40.0, -40.0, 200.0, -200.0, 3e4, -3e4,
                                                                1e18, -1e18, 1e25, -1e25])]).to(t)
    n = gate.numel()
    pre = torch.cat([gate, torch.full((n,), 1.5)]).to(t)[None]
    dh, x, w = torch.full((1, n), 0.75, dtype=t), torch.ones(1, 8, dtype=t), torch.zeros(2 * n, 8, dtype=t)
    got = backward(dh, x, w, pre, act)
    want = ref.gated_backward(dh, x, w, pre, got["dpre"].cpu(), act, dtype, dtype)["dpre"]
    near = (gate.abs() <= 12).repeat(2)[None]
    assert ref.worst(got["dpre"].cpu()[near], want[0][near], want[1][near] + 1e-38) <= 1.0
    far, there = got["dpre"].cpu().double()[~near], want[0][~near]
    # past the activation's bend: the limits, to the type's rounding
    assert bool(((far - there).abs() <= 2 * ref.HALF[dtype] * there.abs() + 1e-14).all())
    # forward, through the bias: x W^T = 0
    h, kept = forward(x, w, pre[0].float(), act)
    assert torch.equal(kept.cpu(), pre)
    assert bool(h.isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_parts_left_out(dtype):
    """No bias, nothing kept, single outputs: the same bits as with all of them."""
    import torch
    x, w, b, pre, dh = inputs(140, 90, 70, dtype)
    h, kept = forward(x, w, b, "silu")
    assert torch.equal(forward(x, w, b, "silu", keep=False)[0], h)
    plain = forward(x, w, None, "silu")
    for got, want in zip(plain, forward(x, w, torch.zeros(140), "silu")):
        assert torch.equal(got, want)
    got = backward(dh, x, w, pre, "gelu")
    at = [t.to(DEV) for t in (dh, x, w, pre)]
    for name in ("dx", "dweight", "dbias"):
        one, dpre = torch.full_like(got[name], float("nan")), torch.full_like(got["dpre"], float("nan"))
        la.kfac_gated_backward(*at, dpre, activation="gelu", **{name: one})
        assert torch.equal(one, got[name]) and torch.equal(dpre, got["dpre"])


def test_weight_gradient_in_float32():
    x, w, b, pre, dh = inputs(150, 66, 130, "bf16")
    import torch
    got = backward(dh, x, w, pre, "silu", dweight_type=torch.float32)
    hold(got, ref.gated_backward(dh, x, w, pre, got["dpre"].cpu(), "silu", "bf16", "f32"))
    assert torch.equal(got["dweight"].bfloat16(), backward(dh, x, w, pre, "silu")["dweight"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(dtype):
    import torch
    x, w, b, pre, dh = inputs(0, 20, 6, dtype)
    assert forward(x, w, b, "relu")[0].shape == (0, 6)
    got = backward(dh, x, w, pre, "relu")
    assert not got["dweight"].any() and not got["dbias"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_memory_around_stays(dtype):
    """Outputs inside larger buffers, unaligned where that is allowed."""
    import torch
    rows, d, width = 131, 77, 45
    x, w, b, pre, dh = inputs(rows, d, width, dtype)
    want_h, want_pre = forward(x, w, b, "silu")
    want = backward(dh, x, w, pre, "silu")
    shapes = {"h": (rows, width), "pre": (rows, 2 * width), "dpre": (rows, 2 * width), "dx": (rows, d), "dweight": (2 * width, d)}
    room = {k: torch.full((s[0] * s[1] + 16,), 5.0, dtype=x.dtype, device=DEV) for k, s in shapes.items()}
    lead = {"h": 1, "pre": 3, "dpre": 4, "dx": 5, "dweight": 7}
    at = {k: room[k][lead[k]:lead[k] + s[0] * s[1]].view(s) for k, s in shapes.items()}
    la.kfac_gated_forward(x.to(DEV), w.to(DEV), at["h"], bias=b.to(DEV), pre=at["pre"])
    db = torch.full((2 * width + 2,), 5.0, device=DEV)
    # inputs that begin on any element too (x and weight on 4 bytes)
    lone = [torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape).copy_(t) for t in (dh, pre)]
    la.kfac_gated_backward(lone[0], x.to(DEV), w.to(DEV), lone[1], at["dpre"], at["dx"], at["dweight"], db[1:-1])
    for name, value in (("h", want_h), ("pre", want_pre), *((k, want[k]) for k in ("dpre", "dx", "dweight"))):
        assert torch.equal(at[name], value), name
        at[name].fill_(5.0)
        assert bool((room[name] == 5.0).all()), name
    assert torch.equal(db[1:-1], want["dbias"]) and float(db[0]) == float(db[-1]) == 5.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_numbers_that_are_none_stay_in_their_rows(dtype):
    """A NaN in one row of x reaches that row's h alone; in dh, that row's dx."""
    import torch
    rows, d, width = 150, 45, 50
    x, w, b, pre, dh = inputs(rows, d, width, dtype)
    h, _ = forward(x, w, b, "gelu")
    got = backward(dh, x, w, pre, "gelu")
    bad, worse = x.clone(), dh.clone()
    bad[77, 44] = worse[20, 49] = float("nan")
    h2, _ = forward(bad, w, b, "gelu")
    again = backward(worse, x, w, pre, "gelu")
    keep = [r for r in range(rows) if r != 77]
    assert torch.equal(h2[keep], h[keep]) and bool(h2[77].isnan().all())
    keep = [r for r in range(rows) if r != 20]
    assert torch.equal(again["dx"][keep], got["dx"][keep]) and bool(again["dx"][20].isnan().all())
    # and one in a column of dpre that column of dweight alone
    rest = [c for c in range(2 * width) if c not in (49, 99)]
    assert torch.equal(again["dweight"][rest], got["dweight"][rest]) and torch.equal(again["dbias"][rest], got["dbias"][rest])


def test_large_float32_values():
    """Numbers past bfloat16's largest keep their size; tiny ones keep theirs."""
    import torch
    x = torch.tensor([[3.4e38, 0.0], [1e-30, 2.0 ** -100]])
    w = torch.tensor([[1e-38, 0.0], [1.0, 1.0], [0.0, 1e-8], [1e-38, 1.0]])
    _, pre = forward(x, w, None, "relu")
    want = x.double() @ w.double().t()
    xa, wa = x.double().abs(), w.double().abs()
    limit = 8 * ref.U32 * (xa @ wa.t()) + 2.0 ** -126
    # parts under 2^-126 may be lost: of each number up to 2^-126 (1 + 2^-8 + 2^-16),
    # which the other factor multiplies (1e-38 lies under 2^-126 itself)
    lost = 2.0 ** -126 * (1 + 2.0 ** -8 + 2.0 ** -16)
    limit = limit + lost * (xa.sum(1)[:, None] + wa.sum(1)[None, :])
    assert bool(((pre.cpu().double() - want).abs() <= limit).all())
    # which leaves the products of the larger numbers their rounding
    assert abs(float(pre[0, 1]) / 3.4e38 - 1) <= 2.0 ** -23 and abs(float(pre[1, 1]) / float(want[1, 1]) - 1) <= 2.0 ** -22


def test_gradients_against_differences():
    import torch
    x, w, b, _, dh = inputs(9, 40, 30, "f32")
    for act in ACTS:
        _, pre = forward(x, w, b, act)
        got = backward(dh, x, w, pre.cpu(), act)
        g = torch.Generator().manual_seed(3)
        way = [torch.randn(*t.shape, generator=g).double() for t in (x, w, b)]
        h = 1e-5

        def value(s):
            at = [t.double() + s * h * v for t, v in zip((x, w, b), way)]
            p = at[0] @ at[1].t() + at[2]
            return float((ref.activation(act, p[:, :30])[0] * p[:, 30:] * dh.double()).sum())

        along = (value(1) - value(-1)) / (2 * h)
        mine = [got[k].double().cpu() for k in ("dx", "dweight", "dbias")]
        there = sum(float((t * v).sum()) for t, v in zip(mine, way))
        size = sum(float((t * v).abs().sum()) for t, v in zip(mine, way))
        # float32 gradients of sums of up to 60 terms; the differences' third order, h^2 times the
        # directions' squares; relu's bend may be crossed by numbers within h |way| of it
        limit = size * (200 * ref.U32 + 1e-7) + (1e-3 * size if act == "relu" else 0.0)
        say(f"  {act} {abs(along - there):.2e} of {limit:.2e}")
        assert abs(along - there) <= limit


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_again_and_on_another_stream(dtype):
    import torch
    x, w, b, pre, dh = (t.to(DEV) for t in inputs(700, 330, 170, dtype))
    got, side = [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side):
        h, kept = nan(700, 170, dtype=x.dtype), nan(700, 340, dtype=x.dtype)
        dpre, dx, dw, db = (torch.empty_like(t) for t in (pre, x, w, b))
        torch.cuda.synchronize()
        la.kfac_gated_forward(x, w, h, bias=b, pre=kept, stream=stream)
        la.kfac_gated_backward(dh, x, w, pre, dpre, dx, dw, db, stream=stream)
        torch.cuda.synchronize()
        got.append((h, kept, dpre, dx, dw, db))
    for other in got[1:]:
        for a, c in zip(got[0], other):
            assert torch.equal(a, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(dtype):
    """Both passes in a graph, replayed on new inputs with eager work between."""
    import torch
    x, w, b, pre, dh = (t.to(DEV) for t in inputs(333, 129, 65, dtype))
    outs = [torch.empty_like(t) for t in (dh, pre, pre, x, w, b)]

    def step():
        la.kfac_gated_forward(x, w, outs[0], bias=b, pre=outs[1])
        la.kfac_gated_backward(dh, x, w, outs[1], outs[2], outs[3], outs[4], outs[5])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(inputs(333, 129, 65, dtype, seed=seed + 1)[0])
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(outs, want):
            assert torch.equal(a, c)
