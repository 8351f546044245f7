"""GPU: the gated feed-forward block at sizes whose products take every way
there is: the largest tiles, a last round shared out, long reductions of few
tiles, few rows against many.  Compared on the GPU with float64 forms."""
import pytest

import linear_algebra_amd as la
from tests import encoder_reference as ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

# 3001 x 3001 x 4101: 256 x 256 tiles, whole and shared ones of both gradients;
# 8200 x 520 x 4100, 8300 x 2000 x 4200: forward by such tiles, all whole and some shared;
# 16390 x 70 x 4096: outputs past the caches; 2304 x 520 x 5000: all of dx shared out
# beside whole tiles of dw; 20001 x 33 x 9: the other way round; the rest: odd
# widths, long sums of one tile, both sides of where few rows end
BF16 = [(3001, 3001, 4101), (8200, 520, 4100), (2304, 520, 5000), (4000, 600, 700), (4100, 2051, 1100), (130, 5001, 260),
        (66, 9001, 33), (2, 16384, 17), (8300, 2000, 4200), (16390, 70, 4096), (64, 1024, 515), (65, 1024, 515), (129, 1024, 515), (20001, 33, 9), (3, 20, 16384)]
F32 = [(1834, 1445, 2031), (1301, 515, 1203), (700, 2049, 500), (64, 2510, 116), (65, 2510, 116), (180, 2510, 116), (300, 16384, 40),
       (20001, 33, 9), (3, 20, 16384), (5000, 200, 300)]
CASES = [("bf16", *s) for s in BF16] + [("f32", *s) for s in F32]


def inputs(dtype, rows, d, width):
    import torch
    g = torch.Generator(device=DEV).manual_seed(rows + 3 * d + 5 * width)
    t = ref.types()[dtype]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    return (normal(rows, d).to(t), (normal(2 * width, d) * d ** -0.5).to(t), normal(2 * width), (normal(rows, 2 * width) * 2).to(t),
            normal(rows, width).to(t))


def worst(got, value, bound):
    """The largest error in units of its bound, where they are."""
    import torch
    err = (got.double() - value).abs()
    ratio = torch.where(err > 0, err / bound.clamp_min(1e-300), torch.zeros_like(err))
    return float(ratio.nan_to_num(nan=float("inf")).max())


def hold(got, want):
    for name, value in got.items():
        r = worst(value, *want[name])
        say(f"  {name} {r:.3f}")
        assert r <= 1.0, name


@pytest.mark.parametrize("dtype,rows,d,width", CASES)
def test_forward(dtype, rows, d, width):
    import torch
    act = list(la.KFAC_ACTIVATIONS)[(rows + d) % 5]
    x, w, b, _, _ = inputs(dtype, rows, d, width)
    h = torch.full((rows, width), float("nan"), dtype=x.dtype, device=DEV)
    pre = torch.full((rows, 2 * width), float("nan"), dtype=x.dtype, device=DEV)
    la.kfac_gated_forward(x, w, h, bias=b, pre=pre, activation=act)
    hold({"h": h, "pre": pre}, ref.gated_forward(x, w, b, act, dtype))
    alone = torch.full_like(h, float("nan"))
    la.kfac_gated_forward(x, w, alone, bias=b, activation=act)
    assert torch.equal(alone, h)


@pytest.mark.parametrize("dtype,rows,d,width", CASES)
def test_backward(dtype, rows, d, width):
    import torch
    act = list(la.KFAC_ACTIVATIONS)[(rows + d + 2) % 5]
    x, w, _, pre, dh = inputs(dtype, rows, d, width)
    got = {"dpre": torch.full_like(pre, float("nan")), "dx": torch.full_like(x, float("nan")),
           "dweight": torch.full_like(w, float("nan")), "dbias": torch.full((2 * width,), float("nan"), device=DEV)}
    la.kfac_gated_backward(dh, x, w, pre, activation=act, **got)
    want = ref.gated_backward(dh, x, w, pre, got["dpre"], act, dtype, dtype)
    hold(got, want)
    # each product by itself, which may share its tiles out otherwise
    for name in ("dx", "dweight"):
        one = torch.full_like(got[name], float("nan"))
        la.kfac_gated_backward(dh, x, w, pre, got["dpre"], activation=act, **{name: one})
        hold({name: one}, want)


@pytest.mark.parametrize("dtype,rows,d,width", [("bf16", 2304, 520, 1500), ("bf16", 130, 5001, 260), ("f32", 700, 1025, 300)])
def test_two_streams_and_a_graph_at_once(dtype, rows, d, width):
    """Passes on two streams while a captured one is replayed on a third, each
    with its own workspace: the bits of each alone."""
    import torch
    sides = [torch.cuda.Stream() for _ in range(2)]
    ins, outs, want = [], [], []
    for k in range(3):
        x, w, b, _, dh = inputs(dtype, rows, d, width + 2 * k)
        ins.append((x, w, b, dh))
        outs.append([torch.empty(rows, width + 2 * k, dtype=x.dtype, device=DEV)] +
                    [torch.empty(rows, 2 * (width + 2 * k), dtype=x.dtype, device=DEV) for _ in range(2)] +
                    [torch.empty_like(t) for t in (x, w, b)])

    def step(k, stream=None):
        x, w, b, dh = ins[k]
        h, pre, dpre, dx, dw, db = outs[k]
        la.kfac_gated_forward(x, w, h, bias=b, pre=pre, stream=stream)
        la.kfac_gated_backward(dh, x, w, pre, dpre, dx, dw, db, stream=stream)

    for k in range(3):
        step(k)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs[k]])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(2)
    for _ in range(3):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(2):
            for k in range(2):
                step(k, sides[k])
            graph.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            for a, c in zip(o, v):
                assert torch.equal(a, c)


def test_most_rows():
    """Row numbers and offsets past 32 bits, to the last rows that a launch can
    have.  Every row holds one of 8 inputs, so that every output is one of 8 numbers."""
    import torch
    rows, whole = 2 ** 31 - 259, 2 ** 31 - 264
    g = torch.Generator(device=DEV).manual_seed(5)
    pick = torch.randn(8, 2, generator=g, device=DEV).bfloat16()
    w = torch.randn(2, 2, generator=g, device=DEV).bfloat16()

    def many(t):
        return t.repeat(2 ** 28, 1)[:rows]

    def holds(got, few):
        n = few.shape[1]
        assert torch.equal(got[:whole * n].view(-1, 8 * n), few.view(1, 8 * n).expand(whole // 8, 8 * n))
        assert torch.equal(got[whole * n:rows * n], few.view(-1)[:(rows - whole) * n]) and bool((got[rows * n:] == 7.0).all())

    room = torch.full((rows + 4096,), 7.0, dtype=torch.bfloat16, device=DEV)
    x = many(pick)
    la.kfac_gated_forward(x, w, room[:rows].view(rows, 1), activation="silu")
    few, pre = torch.empty(8, 1, dtype=x.dtype, device=DEV), torch.empty(8, 2, dtype=x.dtype, device=DEV)
    la.kfac_gated_forward(pick, w, few, pre=pre, activation="silu")
    # sums of two exact products, rounded alike whichever kernel forms them
    holds(room, few)
    del room
    dpre, dx = (torch.full((2 * rows + 4096,), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    la.kfac_gated_backward(many(few), x, w, many(pre), dpre[:2 * rows].view(rows, 2), dx=dx[:2 * rows].view(rows, 2), activation="silu")
    few_dpre, few_dx = torch.empty_like(pre), torch.empty_like(pick)
    la.kfac_gated_backward(few, pick, w, pre, few_dpre, dx=few_dx, activation="silu")
    holds(dpre, few_dpre)
    holds(dx, few_dx)
    # and one more tile is refused
    more = torch.empty(2 ** 31 - 1, 2, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(la.KfacError, match="UNSUPPORTED"):
        la.kfac_gated_forward(more, w, more.view(-1)[:2 ** 31 - 1].view(-1, 1), activation="silu")
