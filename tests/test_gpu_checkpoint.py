"""GPU: layer inputs kept in 8 bits.  Codes and values bit for bit against a
float64 form; the factor and the gradient within float32 summation bounds."""
import numpy as np
import pytest

import linear_algebra_amd as la
from tests import training_reference as ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
TINY = 2.0 ** -126        # float32 products below the smallest normal number may come out as zero

SHAPES = [(1, 1, False), (1, 1, True), (31, 2, True), (32, 3, False), (33, 64, True), (100, 255, True), (128, 1024, True),
          (97, 514, False), (65, 2049, False)]


def inputs(rows, d, dtype, seed):
    import torch
    rng = np.random.default_rng(seed)
    x = np.maximum(rng.standard_normal((rows, d)), -0.5)
    x[:, rng.random(d) < 0.2] *= 100.0
    x[:, rng.random(d) < 0.1] *= 2.0 ** -120
    x[:, rng.random(d) < 0.05] = 0.0
    if d > 2:
        # half steps of the codes: ties
        x[:, 1] = (rng.integers(0, 16, rows) + 0.5) * 2.0 ** rng.integers(-3, 3)
    t = torch.from_numpy(x.astype(np.float32))
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def keep(x, ones):
    codes, scales = la.kfac_checkpoint_empty(x.shape[0], x.shape[1] + int(ones), DEV)
    codes.fill_(0xAA)
    la.kfac_checkpoint_store([x], [codes], [scales], ones=ones)
    return codes, scales


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d,ones", SHAPES)
def test_store_and_load(rows, d, ones, dtype):
    import torch
    x = inputs(rows, d, dtype, rows + d)
    codes, scales = keep(x.to(DEV), ones)
    wc, ws = ref.encode(x.float().numpy(), ones)
    np.testing.assert_array_equal(scales.cpu().numpy(), ws)
    np.testing.assert_array_equal(codes.cpu().numpy(), wc)
    want = ref.decode(wc, ws, rows)
    for t in (torch.bfloat16, torch.float32):
        for cols in {d + int(ones), d, max(1, d // 2)}:
            y = torch.full((rows, cols), float("nan"), dtype=t, device=DEV)
            la.kfac_checkpoint_load([codes], [scales], [y])
            np.testing.assert_array_equal(y.float().cpu().numpy().astype(np.float64), want[:, :cols])


def test_values_at_the_ends_of_the_range():
    """Zero, both infinities, NaN, subnormals, the largest float32 and its neighbours."""
    import torch
    x = np.zeros((64, 8), dtype=np.float32)
    x[3, 0], x[4, 0], x[5, 0], x[6, 0] = np.inf, -np.inf, np.nan, 3.0
    x[:32, 1] = np.float32(2.0 ** -149) * np.arange(32)
    x[:, 2] = -np.float32(0.0)
    x[7, 3], x[8, 3] = np.float32(3.0e38), -np.float32(1.9e38)
    x[:, 4] = 2.0 ** -126 * np.linspace(-1, 1, 64)
    x[:, 5] = 448.0 * np.where(np.arange(64) % 2, 1, -1)
    x[:, 6] = np.nextafter(np.float32(448.0), np.float32(500.0))
    x[:32, 7] = np.inf
    codes, scales = keep(torch.from_numpy(x).to(DEV), False)
    wc, ws = ref.encode(x, False)
    got = codes.cpu().numpy()
    np.testing.assert_array_equal(scales.cpu().numpy(), ws)
    nan = (wc & 0x7f) == 0x7f
    np.testing.assert_array_equal((got & 0x7f) == 0x7f, nan)      # a NaN's sign is free
    np.testing.assert_array_equal(got[~nan], wc[~nan])
    y = torch.empty(64, 8, device=DEV)
    la.kfac_checkpoint_load([codes], [scales], [y])
    y = y.cpu().numpy()
    assert np.array_equal(np.isnan(y), np.isnan(ref.decode(wc, ws, 64)))


def test_unaligned_rows():
    """An input one element off its allocation's start: no 4-byte access may be assumed."""
    import torch
    x = inputs(70, 64, "bf16", 9)
    wide = torch.zeros(70 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    view = wide[1:].view(70, 64)
    view.copy_(x)
    codes, scales = keep(view, True)
    wc, ws = ref.encode(x.float().numpy(), True)
    np.testing.assert_array_equal(codes.cpu().numpy(), wc)
    np.testing.assert_array_equal(scales.cpu().numpy(), ws)


def check(got, want, bound, name):
    err = np.abs(got - want)
    worst = float((err / np.maximum(bound, 1e-300)).max())
    say(f"  {name}: error at most {worst:.3f} of its bound")
    assert np.all(err <= bound), (name, worst)


FACTORS = [(1, 1, False), (5, 33, True), (64, 128, False), (100, 129, True), (333, 300, True), (1000, 257, False),
           (4096, 260, True), (25088, 130, True)]


def test_factors():
    """Every shape in one call (more layers than one launch carries), first step and running average, the
    strict lower triangle left as it was."""
    import torch
    xs = [inputs(r, d, "bf16", r) for r, d, _ in FACTORS]
    kept = [keep(x.to(DEV), o) for x, (_, _, o) in zip(xs, FACTORS)]
    xs = xs + [inputs(40, 20, "bf16", 3)]
    kept = kept + [keep(xs[-1].to(DEV), False)]
    rows = [r for r, _, _ in FACTORS] + [40]
    codes, scales = [c for c, _ in kept], [s for _, s in kept]
    ms = [torch.full((c.shape[1], c.shape[1]), float("nan"), device=DEV) for c in codes]
    la.kfac_checkpoint_factors(codes, scales, rows, ms, 0.9, True)
    first = [m.cpu().numpy().astype(np.float64) for m in ms]
    la.kfac_checkpoint_factors(codes, scales, rows, ms, 0.9, False)
    for c, s, r, m1, m in zip(codes, scales, rows, first, ms):
        x = ref.decode(c.cpu().numpy(), s.cpu().numpy(), r)
        want, mag = x.T @ x / r, np.abs(x).T @ np.abs(x) / r
        up = np.triu_indices(x.shape[1])
        # sums of at most min(rows, 4096) + 64 float32 additions, one scaling
        bound = (min(r, 4096) + 66) * U32 * mag + TINY
        check(m1[up], want[up], bound[up], f"factor {r} x {x.shape[1]}")
        low = np.tril_indices(x.shape[1], -1)
        assert np.all(np.isnan(m1[low]))
        m2 = m.cpu().numpy().astype(np.float64)
        check(m2[up], want[up], (bound + 4 * U32 * np.abs(want))[up], "running average of equal steps")


GRADS = [(1, 1, 1, False), (7, 10, 33, True), (32, 128, 128, False), (33, 130, 257, True), (200, 100, 100, True),
         (128, 1024, 300, True), (1000, 64, 200, True), (4096, 136, 264, False)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients(dtype):
    import torch
    gs, kept, mats = [], [], []
    for r, o, d, ones in GRADS:
        kept.append(keep(inputs(r, d, "bf16", r + d).to(DEV), ones))
        g = torch.randn(r, o, generator=torch.Generator().manual_seed(r)) * 1e-3
        gs.append(g.to(torch.bfloat16) if dtype == "bf16" else g)
        mats.append(torch.full((o, d + int(ones)), float("nan"), device=DEV))
    la.kfac_checkpoint_grad([g.to(DEV) for g in gs], [c for c, _ in kept], [s for _, s in kept], mats)
    for g, (c, s), m in zip(gs, kept, mats):
        r = g.shape[0]
        x, gd = ref.decode(c.cpu().numpy(), s.cpu().numpy(), r), g.double().numpy()
        # three parts per float32 gradient: three additions per row
        bound = ((3 if dtype == "f32" else 1) * r + 16) * U32 * (np.abs(gd).T @ np.abs(x)) + r * TINY
        check(m.cpu().numpy().astype(np.float64), gd.T @ x, bound, f"gradient {r} x {g.shape[1]} x {x.shape[1]}")


def test_gradient_of_unaligned_rows():
    import torch
    kept = keep(inputs(50, 40, "bf16", 1).to(DEV), False)
    for t in (torch.bfloat16, torch.float32):
        wide = torch.randn(50 * 64 + 1, device=DEV).to(t)
        g = wide[1:].view(50, 64)
        a, b = torch.empty(64, 40, device=DEV), torch.empty(64, 40, device=DEV)
        la.kfac_checkpoint_grad([g], [kept[0]], [kept[1]], [a])
        la.kfac_checkpoint_grad([g.clone()], [kept[0]], [kept[1]], [b])
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", [0, 1, 3])
def test_gradient_of_odd_widths(dtype, first):
    """Rows that begin inside a 4-byte word, or in the middle of 16 bytes, between NaN on both sides."""
    import torch
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(11)
    for r, d, m in ((1, 16, 1), (33, 40, 7), (64, 24, 9), (65, 130, 127), (100, 33, 129), (700, 20, 131), (127, 17, 258),
                    (640, 140, 5)):
        say("odd gradient", dtype, first, r, d, m)
        codes, scales = keep(inputs(r, d, "bf16", m).to(DEV), True)
        g = torch.randn(r, m, generator=gen).to(t)
        wide = torch.full((r * m + 8,), float("nan"), dtype=t, device=DEV)
        wide[first:first + r * m] = g.to(DEV).flatten()
        out = torch.full((m, d + 1), float("nan"), device=DEV)
        la.kfac_checkpoint_grad([wide[first:first + r * m].view(r, m)], [codes], [scales], [out])
        x, gd = ref.decode(codes.cpu().numpy(), scales.cpu().numpy(), r), g.double().numpy()
        bound = ((3 if dtype == "f32" else 1) * r + 16) * U32 * (np.abs(gd).T @ np.abs(x)) + r * TINY
        check(out.cpu().numpy().astype(np.float64), gd.T @ x, bound, f"gradient {r} x {m} x {d + 1}")


def test_nan_spreads_to_its_column():
    """A NaN in the input reaches its row and column of the factor and its column of the gradient, nothing else."""
    import torch
    x = inputs(100, 64, "f32", 4)
    x[17, 5] = float("nan")
    codes, scales = keep(x.to(DEV), False)
    m = torch.zeros(64, 64, device=DEV)
    la.kfac_checkpoint_factors([codes], [scales], [100], [m], 0.9, True)
    want = torch.zeros(64, 64, dtype=torch.bool)
    want[5, 5:] = want[:6, 5] = True
    assert torch.equal(torch.isnan(m).cpu(), want)
    mat = torch.zeros(16, 64, device=DEV)
    la.kfac_checkpoint_grad([torch.ones(100, 16, device=DEV)], [codes], [scales], [mat])
    assert torch.equal(torch.isnan(mat).cpu().all(0), torch.arange(64) == 5) and not torch.isnan(mat[:, 6:]).any()


def test_same_bits_on_another_stream_and_in_a_graph():
    import torch
    x = inputs(1000, 300, "bf16", 11).to(DEV)
    g = torch.randn(1000, 77, device=DEV)

    def room():
        c, s = la.kfac_checkpoint_empty(1000, 301, DEV)
        return {"c": c, "s": s, "m": torch.zeros(301, 301, device=DEV), "g": torch.zeros(77, 301, device=DEV),
                "y": torch.zeros(1000, 301, device=DEV)}

    def step(r, stream=None):
        la.kfac_checkpoint_store([x], [r["c"]], [r["s"]], ones=True, stream=stream)
        la.kfac_checkpoint_load([r["c"]], [r["s"]], [r["y"]], stream=stream)
        la.kfac_checkpoint_factors([r["c"]], [r["s"]], [1000], [r["m"]], 0.9, True, stream=stream)
        la.kfac_checkpoint_grad([g], [r["c"]], [r["s"]], [r["g"]], stream=stream)

    eager, other, cap = room(), room(), room()
    step(eager)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(other, side)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for n in eager:
        assert torch.equal(eager[n], other[n]), n
    for replay in range(3):
        x.copy_(inputs(1000, 300, "bf16", 20 + replay))
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for n in eager:
            assert torch.equal(eager[n], cap[n]), (replay, n)


def test_gradients_at_the_ends_of_float32():
    """Infinities and NaN reach the rows they belong to as they are, the
    largest numbers (past bfloat16's) stay finite, and the smallest lose what
    lies under bfloat16's subnormals at most: two parts, each below 2^-126."""
    import torch
    rows, d, m = 70, 40, 24
    x = np.random.default_rng(3).uniform(0.5, 1.0, (rows, d)) * 2.0 ** -8
    codes, scales = keep(torch.from_numpy(x.astype(np.float32)).to(DEV), True)
    xh = ref.decode(codes.cpu().numpy(), scales.cpu().numpy(), rows)
    assert np.all(xh > 0)
    top = float(torch.finfo(torch.float32).max)
    g = torch.randn(rows, m, generator=torch.Generator().manual_seed(4))
    g[5, 0], g[9, 1] = float("inf"), -float("inf")
    g[3, 2], g[60, 2] = float("inf"), -float("inf")          # cancel to NaN
    g[69, 3] = float("nan")
    g[:, 4] = 0.0
    g[0, 4], g[1, 4], g[40, 4] = top, -top * (1 - 2.0 ** -9), 3.3961775e38
    g[:, 5] *= 2.0 ** -100
    g[:, 6] *= 2.0 ** -115
    g[:, 7] *= 2.0 ** -126
    g[:, 8] *= 2.0 ** 120
    mat = torch.full((m, d + 1), float("nan"), device=DEV)
    la.kfac_checkpoint_grad([g.to(DEV)], [codes], [scales], [mat])
    gd = g.double().numpy()
    with np.errstate(invalid="ignore"):
        want = gd.T @ xh
    got = mat.cpu().numpy().astype(np.float64)
    got, want = got[:, :d], want[:, :d]                     # (the column of ones adds the largest numbers: infinite)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    fin = np.isfinite(want)
    mag = np.abs(np.where(np.isfinite(gd), gd, 0.0)).T @ np.abs(xh)
    # three parts per gradient: three additions per row
    bound = (3 * rows + 16) * U32 * mag + 2.0 ** -125 * np.abs(xh).sum(0) + rows * TINY
    check(got[fin], want[fin], bound[:, :d][fin], "gradients at the ends of float32")
