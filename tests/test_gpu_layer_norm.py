"""GPU: layer norm forward and backward against float64 forms, elementwise
within what the formulas' roundings allow."""
import pytest

import linear_algebra_amd as la
from tests import encoder_reference as ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

# one element, less than a vector, whole and broken vectors, both sides of every form's longest row
SHAPES = [(1, 1), (5, 1), (3, 2), (1, 3), (6, 7), (7, 8), (4, 9), (33, 64), (2, 65), (9, 511), (9, 512), (9, 513), (5, 1023),
          (5, 1024), (5, 1025), (3, 2048), (3, 2049), (3, 4095), (3, 4096), (2, 4097), (2, 8192), (2, 8193), (1, 16383),
          (1, 16384), (700, 1000), (2500, 129), (1300, 2305), (600, 5000), (31, 63), (100, 127), (71, 128), (41, 255), (19, 256),
          (23, 257), (20001, 40), (5003, 100), (4099, 200), (20003, 5), (5, 6144), (5, 6145), (600, 7001)]
FORMS = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


def inputs(rows, d, dtype, weight_dtype, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed + 7 * rows + d)
    t, wt = ref.types()[dtype], ref.types()[weight_dtype]

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    x = (normal(rows, d) * torch.exp(normal(rows, 1)) + normal(rows, 1)).to(t)
    return x, normal(rows, d).to(t), (1 + 0.3 * normal(d)).to(wt), normal(d).to(wt)


def forward(x, w, b, eps=1e-5, stats=True):
    import torch
    x = x.to(DEV)
    y = torch.full_like(x, float("nan"))
    mean, rstd = (torch.full((x.shape[0],), float("nan"), device=DEV) for _ in range(2))
    w, b = (None if t is None else t.to(DEV) for t in (w, b))
    la.kfac_layer_norm_forward(x, y, *((mean, rstd) if stats else ()), weight=w, bias=b, eps=eps)
    return y, mean, rstd


@pytest.mark.parametrize("dtype,weight_dtype", FORMS)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward_and_backward(rows, d, dtype, weight_dtype):
    import torch
    x, dy, w, b = inputs(rows, d, dtype, weight_dtype)
    y, mean, rstd = forward(x, w, b)
    want = ref.norm_forward(x, w, b, 1e-5, dtype)
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        r = ref.worst(got, *want[name])
        say(f"  {name} {r:.3f}")
        assert r <= 1.0, name
    dx = torch.full((rows, d), float("nan"), dtype=x.dtype, device=DEV)
    dw, db = (torch.full((d,), float("nan"), dtype=w.dtype, device=DEV) for _ in range(2))
    la.kfac_layer_norm_backward(dy.to(DEV), x.to(DEV), mean, rstd, dx, weight=w.to(DEV), dweight=dw, dbias=db)
    want = ref.norm_backward(dy, x, mean.cpu(), rstd.cpu(), w, dtype, weight_dtype)
    for name, got in (("dx", dx), ("dweight", dw), ("dbias", db)):
        r = ref.worst(got, *want[name])
        say(f"  {name} {r:.3f}")
        assert r <= 1.0, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_left_out(dtype):
    """No weight, no bias, no statistics, single outputs: the same bits as with all of them."""
    import torch
    x, dy, w, b = inputs(40, 300, dtype, "f32")
    y, mean, rstd = forward(x, w, b)
    assert torch.equal(y, forward(x, w, b, stats=False)[0])
    plain, _, _ = forward(x, None, None)
    assert torch.equal(plain, forward(x, torch.ones(300), torch.zeros(300))[0])
    for weight, bias in ((w, None), (None, b)):
        r = ref.worst(forward(x, weight, bias)[0], *ref.norm_forward(x, weight, bias, 1e-5, dtype)["y"])
        assert r <= 1.0
    x, dy, w = x.to(DEV), dy.to(DEV), w.to(DEV)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    la.kfac_layer_norm_backward(dy, x, mean, rstd, dx, weight=w, dweight=dw, dbias=db)
    for name, want in (("dx", dx), ("dweight", dw), ("dbias", db)):
        got = torch.full_like(want, float("nan"))
        la.kfac_layer_norm_backward(dy, x, mean, rstd, weight=w, **{name: got})
        assert torch.equal(got, want), name
    one = torch.empty_like(x)
    la.kfac_layer_norm_backward(dy, x, mean, rstd, one, weight=torch.ones_like(w))
    la.kfac_layer_norm_backward(dy, x, mean, rstd, dx)
    assert torch.equal(one, dx)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [5, 64, 777, 1030, 4100])
def test_strides_and_alignment(dtype, d):
    """Rows of a wider buffer that begin on any element: the same bits, and
    what lies between and behind the rows stays as it was."""
    import torch
    t = ref.types()[dtype]
    x, dy, w, b = inputs(11, d, dtype, "f32")
    y, mean, rstd = forward(x, w, b)
    dx, dw, db = torch.empty(11, d, dtype=t, device=DEV), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    la.kfac_layer_norm_backward(dy.to(DEV), x.to(DEV), mean, rstd, dx, weight=w.to(DEV), dweight=dw, dbias=db)
    for lead, gap in ((1, 0), (3, 5), (0, 7)):
        def wide(v=None):
            buf = torch.full((13 * (d + gap) + lead,), 77.0, dtype=t, device=DEV)
            view = buf[lead:lead + 11 * (d + gap)].view(11, d + gap)[:, :d]
            if v is not None:
                view.copy_(v)
            return buf, view

        (_, vx), (_, vdy), (by, vy), (bdx, vdx) = wide(x), wide(dy), wide(), wide()
        m2, r2 = torch.empty(11, device=DEV), torch.empty(11, device=DEV)
        shifted = torch.zeros(3 * d + 3, device=DEV)
        vw, vb, vdw = (shifted[k * d + 1:(k + 1) * d + 1] for k in range(3))
        vw.copy_(w), vb.copy_(b)
        la.kfac_layer_norm_forward(vx, vy, m2, r2, weight=vw, bias=vb)
        db2 = torch.empty_like(db)
        la.kfac_layer_norm_backward(vdy, vx, m2, r2, vdx, weight=vw, dweight=vdw, dbias=db2)
        for got, want in ((vy, y), (m2, mean), (r2, rstd), (vdx, dx), (vdw, dw), (db2, db)):
            assert torch.equal(got, want)
        for buf, view in ((by, vy), (bdx, vdx)):
            view.fill_(77.0)
            assert bool((buf == 77.0).all())


def test_no_rows():
    import torch
    e, f = torch.empty(0, 50, device=DEV), torch.empty(0, device=DEV)
    la.kfac_layer_norm_forward(e, e.clone(), f, f.clone(), weight=torch.ones(50, device=DEV))
    dw, db = torch.full((50,), 3.0, device=DEV), torch.full((50,), 3.0, device=DEV)
    la.kfac_layer_norm_backward(e, e.clone(), f, f.clone(), e.clone(), dweight=dw, dbias=db)
    assert not dw.any() and not db.any()


def test_mean_far_from_zero():
    """The variance is summed around the mean: a shift of 2^12 standard
    deviations costs the bits that the inputs' own rounding costs."""
    import torch
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 900, generator=g) + 4096.0
    y, mean, rstd = forward(x, None, None)
    want = ref.norm_forward(x, None, None, 1e-5, "f32")
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        assert ref.worst(got, *want[name]) <= 1.0
    flat = torch.full((3, 77), 5.0)
    y, mean, rstd = forward(flat, None, torch.arange(77.0), eps=1e-2)
    assert torch.equal(y.cpu(), torch.arange(77.0).expand(3, 77)) and bool((mean == 5.0).all())


def test_numbers_that_are_none_stay_in_their_rows():
    import torch
    x, dy, w, b = inputs(70, 130, "f32", "f32")
    y, mean, rstd = forward(x, w, b)
    bad = x.clone()
    bad[3, 7], bad[64, 129] = float("nan"), float("inf")
    y2, mean2, rstd2 = forward(bad, w, b)
    keep = [r for r in range(70) if r not in (3, 64)]
    assert torch.equal(y2[keep], y[keep]) and torch.equal(rstd2[keep], rstd[keep])
    assert bool(y2[[3, 64]].isnan().all())
    dx, dx2 = torch.empty(70, 130, device=DEV), torch.empty(70, 130, device=DEV)
    la.kfac_layer_norm_backward(dy.to(DEV), x.to(DEV), mean, rstd, dx, weight=w.to(DEV))
    la.kfac_layer_norm_backward(dy.to(DEV), bad.to(DEV), mean2, rstd2, dx2, weight=w.to(DEV))
    assert torch.equal(dx2[keep], dx[keep]) and bool(dx2[[3, 64]].isnan().all())


def test_gradient_against_differences():
    """dx from differences of the float64 form: one direction, steps of 1e-4."""
    import torch
    x, dy, w, b = inputs(5, 90, "f32", "f32")
    _, mean, rstd = forward(x, w, b)
    dx, dw, db = torch.empty(5, 90, device=DEV), torch.empty(90, device=DEV), torch.empty(90, device=DEV)
    la.kfac_layer_norm_backward(dy.to(DEV), x.to(DEV), mean, rstd, dx, weight=w.to(DEV), dweight=dw, dbias=db)
    g = torch.Generator().manual_seed(2)
    way = [torch.randn(*t.shape, generator=g).double() for t in (x, w, b)]
    h = 1e-4

    def value(s):
        at = [t.double() + s * h * v for t, v in zip((x, w, b), way)]
        c = at[0] - at[0].mean(1, keepdim=True)
        y = c * (c.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * at[1] + at[2]
        return float((y * dy.double()).sum())

    along = (value(1) - value(-1)) / (2 * h)
    got = sum(float((t.double().cpu() * v).sum()) for t, v in zip((dx, dw, db), way))
    size = sum(float((t.double().cpu() * v).abs().sum()) for t, v in zip((dx, dw, db), way))
    # third derivatives times h^2 / 6, in rows of spread 1 / rstd, and the float32 gradients' own roundings
    limit = size * (float((way[0].abs().max() * rstd.cpu().max() * h) ** 2) * 10 + 100 * ref.U32)
    say(f"  {abs(along - got):.2e} of {limit:.2e}")
    assert abs(along - got) <= limit


def test_same_bits_again_and_on_another_stream():
    import torch
    x, dy, w, b = (t.to(DEV) for t in inputs(3000, 700, "bf16", "f32"))
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []
    for stream in (None, side, side):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd, dw, db = (torch.empty(n, device=DEV) for n in (3000, 3000, 700, 700))
        torch.cuda.synchronize()
        la.kfac_layer_norm_forward(x, y, mean, rstd, weight=w, bias=b, stream=stream)
        la.kfac_layer_norm_backward(dy, x, mean, rstd, dx, weight=w, dweight=dw, dbias=db, stream=stream)
        torch.cuda.synchronize()
        got.append((y, mean, rstd, dx, dw, db))
    for other in got[1:]:
        for a, c in zip(got[0], other):
            assert torch.equal(a, c)


def test_captured_and_replayed():
    """Both passes in a graph, replayed on new inputs with eager work between."""
    import torch
    x, dy, w, b = (t.to(DEV) for t in inputs(900, 1500, "f32", "f32"))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, dw, db = (torch.empty(n, device=DEV) for n in (900, 900, 1500, 1500))

    def step():
        la.kfac_layer_norm_forward(x, y, mean, rstd, weight=w, bias=b)
        la.kfac_layer_norm_backward(dy, x, mean, rstd, dx, weight=w, dweight=dw, dbias=db)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (y, mean, rstd, dx, dw, db)
    for seed in range(3):
        x.copy_(inputs(900, 1500, "f32", "f32", seed=seed + 1)[0])
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(outs, want):
            assert torch.equal(a, c)


@pytest.mark.parametrize("rows,d", [(2 ** 31 - 1, 2), (2 ** 20 + 1, 4100)])
def test_offsets_past_32_bits(rows, d):
    """Every row is one of 8: the bits of those alone, and nothing behind the last."""
    import torch
    g = torch.Generator(device=DEV).manual_seed(d)
    x, dy = (torch.randn(8, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    w = torch.randn(d, generator=g, device=DEV)
    whole = rows // 8 * 8

    def many(t):
        return t.repeat(rows // 8 + 1, 1)[:rows]

    def holds(got, few):
        assert torch.equal(got[:whole].view(-1, 8, d), few.expand(whole // 8, 8, d))
        assert torch.equal(got[whole:rows], few[:rows - whole]) and bool((got[rows:] == 7.0).all())

    few, few_dx = torch.empty_like(x), torch.empty_like(x)
    m, r = torch.empty(8, device=DEV), torch.empty(8, device=DEV)
    la.kfac_layer_norm_forward(x, few, m, r, weight=w)
    la.kfac_layer_norm_backward(dy, x, m, r, few_dx, weight=w)
    room = torch.full((rows + 8, d), 7.0, dtype=torch.bfloat16, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    xs = many(x)
    la.kfac_layer_norm_forward(xs, room[:rows], mean, rstd, weight=w)
    holds(room, few)
    assert torch.equal(mean[:whole].view(-1, 8), m.expand(whole // 8, 8)) and torch.equal(rstd[whole:], r[:rows - whole])
    room.fill_(7.0)
    la.kfac_layer_norm_backward(many(dy), xs, mean, rstd, room[:rows], weight=w)
    holds(room, few_dx)
