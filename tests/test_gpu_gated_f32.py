"""GPU: the gated backward pass of bfloat16 rows with a float32 dpre: nothing
between the inputs and the gradients is rounded to bfloat16."""
import pytest

import linear_algebra_amd as la
from tests import encoder_reference as ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu

ACTS = list(la.KFAC_ACTIVATIONS)
# one of each; both sides of vectors, blocks and tiles; odd widths of x; shared tiles of one product and of both
SHAPES = [(1, 1, 1), (1, 8, 2), (2, 3, 5), (3, 16, 7), (15, 40, 16), (17, 130, 97), (33, 65, 63), (64, 70, 64), (127, 129, 127),
          (130, 250, 66), (300, 72, 1), (70, 2, 260), (513, 34, 21), (1100, 260, 390), (20001, 33, 9), (5, 1000, 300),
          (2304, 520, 1500)]


def inputs(rows, d, width, seed=0):
    import torch
    g = torch.Generator(device=DEV).manual_seed(seed + 31 * rows + 7 * d + width)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    return (normal(rows, width).bfloat16(), normal(rows, d).bfloat16(), (normal(2 * width, d) * d ** -0.5).bfloat16(),
            (normal(rows, 2 * width) * 2).bfloat16())


def outputs(rows, d, width, dweight_type=None):
    import torch
    kinds = {"dpre": ((rows, 2 * width), torch.float32), "dx": ((rows, d), torch.bfloat16),
             "dweight": ((2 * width, d), dweight_type or torch.float32), "dbias": ((2 * width,), torch.float32)}
    return {k: torch.full(s, float("nan"), dtype=t, device=DEV) for k, (s, t) in kinds.items()}


def want(dh, x, w, pre, act, dweight_type):
    """{name: (value, bound)} from the inputs alone: dpre's error in float32
    goes through the products, which round as float32 sums do."""
    import torch
    n = w.shape[0] // 2
    p, e = ref.gated_backward(dh, x, w, pre, torch.zeros_like(pre), act, "f32", "f32")["dpre"]
    res = {"dpre": (p, e)}
    for name, a, b, ea, half in (("dx", p, w.double(), e, "bf16"), ("dweight", p.t(), x.double(), e.t(), dweight_type)):
        value, sums = ref.product(a, b, "f32")
        res[name] = value, ea @ b.abs() + sums + ref.HALF[half] * value.abs()
    depth = dh.shape[0] + 64
    res["dbias"] = p.sum(0), e.sum(0) + depth * ref.U32 * p.abs().sum(0)
    assert p.shape[1] == 2 * n
    return res


def hold(got, limits):
    import torch
    for name, value in got.items():
        err = (value.double() - limits[name][0]).abs()
        ratio = torch.where(err > 0, err / limits[name][1].clamp_min(1e-300), torch.zeros_like(err))
        r = float(ratio.nan_to_num(nan=float("inf")).max()) if err.numel() else 0.0
        say(f"  {name} {r:.3f}")
        assert r <= 1.0, name


@pytest.mark.parametrize("rows,d,width", SHAPES)
def test_backward(rows, d, width):
    import torch
    act = ACTS[(rows + d) % len(ACTS)]
    dh, x, w, pre = inputs(rows, d, width)
    got = outputs(rows, d, width)
    la.kfac_gated_backward(dh, x, w, pre, activation=act, **got)
    limits = want(dh, x, w, pre, act, "f32")
    hold(got, limits)
    # the weight's gradient in bfloat16: the same sums, rounded; each output by itself
    low = outputs(rows, d, width, torch.bfloat16)
    la.kfac_gated_backward(dh, x, w, pre, activation=act, **low)
    assert torch.equal(low["dweight"], got["dweight"].bfloat16())
    for name in ("dx", "dweight", "dbias"):
        one = outputs(rows, d, width)
        la.kfac_gated_backward(dh, x, w, pre, one["dpre"], activation=act, **{name: one[name]})
        assert torch.equal(one["dpre"], got["dpre"])
        hold({name: one[name]}, limits)


@pytest.mark.parametrize("rows,d,width", [(100, 40, 50), (3, 4, 900)])
def test_the_rounding_is_the_callers_choice(rows, d, width):
    """With a bfloat16 dpre the products take it as rounded, and that costs
    more than the float32 form's whole bound; its own dpre is the float32 one, rounded."""
    import torch
    dh, x, w, pre = inputs(rows, d, width)
    got, low = outputs(rows, d, width), outputs(rows, d, width)
    low["dpre"] = low["dpre"].bfloat16()
    for o in (got, low):
        la.kfac_gated_backward(dh, x, w, pre, activation="silu", **o)
    assert torch.equal(low["dpre"], got["dpre"].bfloat16()) and torch.equal(low["dbias"], got["dbias"])
    limits = want(dh, x, w, pre, "silu", "f32")
    far = (low["dweight"].double() - limits["dweight"][0]).abs()
    assert float((far / limits["dweight"][1]).max()) > 4.0
    near = (got["dweight"].double() - limits["dweight"][0]).abs()
    assert float(near.norm()) <= 2.0 ** -6 * float(far.norm())


def test_no_rows_and_numbers_that_are_none():
    import torch
    got = outputs(0, 20, 6)
    la.kfac_gated_backward(*inputs(0, 20, 6), activation="relu", **got)
    assert not got["dweight"].any() and not got["dbias"].any()
    dh, x, w, pre = inputs(150, 45, 50)
    got, again = outputs(150, 45, 50), outputs(150, 45, 50)
    la.kfac_gated_backward(dh, x, w, pre, activation="gelu", **got)
    dh[20, 49] = float("nan")
    la.kfac_gated_backward(dh, x, w, pre, activation="gelu", **again)
    rows, cols = [r for r in range(150) if r != 20], [c for c in range(100) if c not in (49, 99)]
    assert torch.equal(again["dx"][rows], got["dx"][rows]) and bool(again["dx"][20].isnan().all())
    assert torch.equal(again["dweight"][cols], got["dweight"][cols]) and torch.equal(again["dbias"][cols], got["dbias"][cols])


def test_memory_around_stays():
    """Outputs inside larger buffers that begin on any element (dpre's: any
    word): the same bits, and nothing beside them."""
    import torch
    rows, d, width = 131, 77, 45
    args = inputs(rows, d, width)
    want_ = outputs(rows, d, width)
    la.kfac_gated_backward(*args, activation="silu", **want_)
    lead = {"dpre": 3, "dx": 5, "dweight": 7, "dbias": 1}
    room = {k: torch.full((t.numel() + 16,), 5.0, dtype=t.dtype, device=DEV) for k, t in want_.items()}
    at = {k: room[k][lead[k]:lead[k] + t.numel()].view(t.shape) for k, t in want_.items()}
    la.kfac_gated_backward(*args, activation="silu", **at)
    for name in want_:
        assert torch.equal(at[name], want_[name]), name
        at[name].fill_(5.0)
        assert bool((room[name] == 5.0).all()), name


def test_captured_and_replayed():
    import torch
    dh, x, w, pre = inputs(333, 129, 65)
    outs = outputs(333, 129, 65)

    def step(stream=None):
        la.kfac_gated_backward(dh, x, w, pre, activation="gelu", stream=stream, **outs)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        dh.copy_(inputs(333, 129, 65, seed=seed + 1)[0])
        step()
        torch.cuda.synchronize()
        kept = {k: t.clone() for k, t in outs.items()}
        for run in (graph.replay, lambda: step(torch.cuda.Stream())):
            for t in outs.values():
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert all(torch.equal(outs[k], kept[k]) for k in outs)


def test_training_layers_choice():
    """A layer that asks for it gets these gradients; its hooks the rounded one."""
    import torch
    from linear_algebra_amd.training import GatedLinear
    torch.manual_seed(0)
    plain, full = (GatedLinear(40, 33, activation="gelu", unrounded=u).to(DEV) for u in (False, True))
    full.load_state_dict(plain.state_dict())
    seen = []
    full.output_grad_hooks.append(lambda m, g: seen.append(g))
    dh, x, _, _ = inputs(70, 40, 33)
    grads = []
    for layer in (plain, full):
        a = x.clone().requires_grad_()
        layer(a).backward(dh)
        grads.append((a.grad, layer.weight.grad, layer.bias.grad))
    w, b = full.weight.detach().bfloat16(), full.bias.detach()
    h, pre = torch.empty_like(dh), torch.empty(70, 66, dtype=x.dtype, device=DEV)
    la.kfac_gated_forward(x, w, h, bias=b, pre=pre, activation="gelu")
    got = outputs(70, 40, 33)
    la.kfac_gated_backward(dh, x, w, pre, activation="gelu", **got)
    for a, c in zip(grads[1], (got["dx"], got["dweight"], got["dbias"])):
        assert torch.equal(a, c)
    assert torch.equal(seen[0], got["dpre"].bfloat16())
    assert not torch.equal(grads[0][1], grads[1][1])
