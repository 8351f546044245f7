"""GPU: the gated forward product by tiles (many rows), whole ones and ones
shared out along the reduction: outputs at any address, what is left out,
memory around them, numbers that are none, graphs and streams."""
import pytest

import linear_algebra_amd as la
from tests import encoder_reference as ref
from tests.gpu_helpers import DEV
from tests.test_gpu_gated_large import hold, inputs

pytestmark = pytest.mark.gpu

# type, rows (past those that the kernel for few rows takes), d, width, whether tiles are shared out
CASES = [("bf16", 4100, 78, 46, False), ("bf16", 4111, 77, 45, False), ("bf16", 4100, 2052, 46, True), ("bf16", 5000, 2051, 45, True),
         ("f32", 4100, 77, 45, False), ("f32", 4111, 78, 46, False), ("f32", 4100, 2052, 46, True), ("f32", 4103, 1001, 131, True)]


def shares(dtype, rows, d, width):
    """Whether a call's workspace holds more than the operands' copies."""
    align = lambda n, a: (n + a - 1) // a * a  # noqa: E731
    copies = 0 if dtype == "bf16" and d % 2 == 0 else 1 if dtype == "bf16" else 3
    held = sum(align(2 * copies * n * align(d, 8), 256) for n in (rows, 2 * width))
    have = la.load_library().kfac_gated_workspace_size(rows, d, width, la.KFAC_BF16 if dtype == "bf16" else la.KFAC_F32, 0)
    assert have >= held
    return have > held


def forward(x, w, b, act="gelu", keep=True, stream=None):
    import torch
    rows, width = x.shape[0], w.shape[0] // 2
    h = torch.full((rows, width), float("nan"), dtype=x.dtype, device=DEV)
    pre = torch.full((rows, 2 * width), float("nan"), dtype=x.dtype, device=DEV) if keep else None
    torch.cuda.synchronize()
    la.kfac_gated_forward(x, w, h, bias=b, pre=pre, activation=act, stream=stream)
    return h, pre


@pytest.mark.parametrize("dtype,rows,d,width,shared", CASES)
def test_values_and_parts_left_out(dtype, rows, d, width, shared):
    import torch
    assert shares(dtype, rows, d, width) == shared
    x, w, b, _, _ = inputs(dtype, rows, d, width)
    for act in la.KFAC_ACTIVATIONS:
        h, pre = forward(x, w, b, act)
        hold({"h": h, "pre": pre}, ref.gated_forward(x, w, b, act, dtype))
        assert torch.equal(forward(x, w, b, act, keep=False)[0], h)
    for got, want in zip(forward(x, w, None), forward(x, w, torch.zeros_like(b))):
        assert torch.equal(got, want)
    hold(dict(zip(("h", "pre"), forward(x, w, None))), ref.gated_forward(x, w, None, "gelu", dtype))


@pytest.mark.parametrize("dtype,rows,d,width,shared", CASES)
@pytest.mark.parametrize("lead", [1, 3])
def test_any_address_and_memory_around(dtype, rows, d, width, shared, lead):
    """Outputs, and the bias, that begin on any element: the same bits, and
    nothing in front of or behind them is written."""
    import torch
    x, w, b, _, _ = inputs(dtype, rows, d, width)
    h, pre = forward(x, w, b)
    room = [torch.full((t.numel() + 4096,), 5.0, dtype=t.dtype, device=DEV) for t in (h, pre)]
    at = [r[lead + 6 * k:lead + 6 * k + t.numel()].view(t.shape) for k, (r, t) in enumerate(zip(room, (h, pre)))]
    shifted = torch.zeros(2 * width + 1, device=DEV)[1:].copy_(b)
    la.kfac_gated_forward(x, w, at[0], bias=shifted, pre=at[1], activation="gelu")
    for r, v, t in zip(room, at, (h, pre)):
        assert torch.equal(v, t)
        v.fill_(5.0)
        assert bool((r == 5.0).all())


@pytest.mark.parametrize("dtype,rows,d,width,shared", CASES)
def test_numbers_that_are_none_stay(dtype, rows, d, width, shared):
    """In their row of x, in their column of the weights."""
    import torch
    x, w, b, _, _ = inputs(dtype, rows, d, width)
    _, pre = forward(x, w, b)
    x[rows - 1, d - 1] = x[129, 0] = float("nan")
    w[width + 5, d - 1] = float("nan")
    h, got = forward(x, w, b)
    keep = [r for r in range(rows) if r not in (129, rows - 1)]
    cols = [c for c in range(2 * width) if c != width + 5]
    assert torch.equal(got[keep][:, cols], pre[keep][:, cols])
    assert bool(got[[129, rows - 1]].isnan().all()) and bool(got[:, width + 5].isnan().all())
    assert bool(h[keep][:, [c for c in range(width) if c != 5]].isfinite().all()) and bool(h[[129, rows - 1]].isnan().all())


@pytest.mark.parametrize("dtype,rows,d,width,shared", [c for c in CASES if c[2] % 2 == 1 or c[4]])
def test_replayed_beside_other_streams(dtype, rows, d, width, shared):
    """A captured pass replayed while two others run on streams of their own,
    each with its own workspace: the bits of each alone, every time."""
    import torch
    x, w, b, _, _ = inputs(dtype, rows, d, width)
    ins = [(x * s).contiguous() for s in (1.0, 0.5, 2.0)]
    want = [forward(v, w, b) for v in ins]
    outs = [[torch.empty_like(t) for t in o] for o in want]
    sides = [torch.cuda.Stream() for _ in range(2)]

    def step(k, stream=None):
        la.kfac_gated_forward(ins[k], w, outs[k][0], bias=b, pre=outs[k][1], activation="gelu", stream=stream)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(2)
    for _ in range(3):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for k in range(2):
                step(k, sides[k])
            graph.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            for a, c in zip(o, v):
                assert torch.equal(a, c)
