"""GPU: the norm of many gradients and their clipping, against float64."""
import math

import pytest

import linear_algebra_amd as la
from tests import encoder_reference as ref
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def gradients(sizes, dtypes, seed=0, lead=0):
    """Views one behind another in a buffer per type, the first `lead` elements in."""
    import torch
    g = torch.Generator().manual_seed(seed)
    got = []
    for k, n in enumerate(sizes):
        t = ref.types()[dtypes[k % len(dtypes)]]
        buf = torch.zeros(lead + n, dtype=t, device=DEV)
        buf[lead:] = torch.randn(n, generator=g).mul_(math.exp(k % 5)).to(DEV).to(t)
        got.append(buf[lead:])
    return got


def norm_of(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


def check(grads, max_norm, outs=None):
    """The norm to a rounding of float32, the outputs to one of the factor, one of the product and one of their type."""
    import torch
    before = [t.clone() for t in grads]
    want = norm_of(grads)
    norm = torch.full((1,), float("nan"), device=DEV)
    la.kfac_grad_norm(grads, norm)
    assert abs(float(norm) - want) <= 1.01 * ref.U32 * want
    again = torch.full((1,), float("nan"), device=DEV)
    la.kfac_grad_clip(grads, max_norm, again, outs=outs)
    assert torch.equal(norm, again)
    c = min(1.0, max_norm / (want + 1e-6))
    for a, o in zip(before, grads if outs is None else outs):
        exact = a.double() * c
        half = ref.HALF["bf16" if a.dtype == torch.bfloat16 else "f32"]
        # the least numbers of both types: their steps are 2^-149 and 2^-133
        limit = exact.abs() * (half + 2.01 * ref.U32) + (2.0 ** -133 if a.dtype == torch.bfloat16 else 2.0 ** -149)
        assert bool(((o.double() - exact).abs() <= limit).all())
        if c == 1.0:
            assert torch.equal(o, a)
    if outs is not None:
        for a, g in zip(before, grads):
            assert torch.equal(a, g)


SETS = [[1], [0, 3], [7, 0, 1, 0], [8191], [8192], [8193, 1, 16384], [5, 100003, 64, 31], [3] * 159, [3] * 160, [3] * 161,
        [17, 0] * 200, [40000] + [9] * 400, [3000000, 11]]


@pytest.mark.parametrize("lead", [0, 1, 3])
@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("bf16", "f32", "f32")], ids="-".join)
@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip(sizes, dtypes, lead):
    import torch
    for share in (0.37, 3.0):
        grads = gradients(sizes, dtypes, seed=len(sizes), lead=lead)
        check(grads, share * norm_of(grads), [torch.full_like(t, float("nan")) for t in grads])
        check(grads, share * norm_of(grads))


def test_extreme_values():
    import torch
    tiny = [torch.full((1000,), 2.0 ** -140, device=DEV), torch.full((24,), 2.0 ** -120, device=DEV)]
    check(tiny, 2.0 ** -119)
    huge = [torch.full((64,), 1e38, device=DEV), torch.full((64,), -3e38, device=DEV, dtype=torch.bfloat16)]
    norm = torch.empty(1, device=DEV)
    la.kfac_grad_clip(huge, 1.0, norm)        # a norm past float32's largest number still scales to 1
    assert math.isinf(float(norm)) and abs(norm_of(huge) - 1.0) <= 2.0 ** -8
    grads = gradients([50, 60], ("f32",))
    check(grads, 0.0)
    assert not any(t.any() for t in grads)
    grads = gradients([50, 60], ("f32",))
    check(grads, float("inf"))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_norms_that_are_no_number(bad):
    """As the formula says: what an infinite norm scales is 0, or NaN where it was infinite; NaN makes all NaN."""
    import torch
    grads = gradients([9000, 70], ("f32", "bf16"))
    grads[1][3] = bad
    norm = torch.empty(1, device=DEV)
    la.kfac_grad_clip(grads, 1.0, norm)
    if math.isinf(bad):
        assert math.isinf(float(norm)) and not grads[0].any() and bool(grads[1][3].isnan())
        assert not grads[1][:3].any() and not grads[1][4:].any()
    else:
        assert math.isnan(float(norm)) and all(bool(t.isnan().all()) for t in grads)


def test_nothing_to_clip():
    import torch
    norm = torch.full((1,), 5.0, device=DEV)
    la.kfac_grad_clip([torch.empty(0, device=DEV)], 1.0, norm)
    assert float(norm) == 0.0
    zeros = [torch.zeros(10000, device=DEV), torch.zeros(3, device=DEV, dtype=torch.bfloat16)]
    la.kfac_grad_clip(zeros, 1.0, norm)
    assert float(norm) == 0.0 and not zeros[0].any()


def test_overlaps_are_refused():
    import torch
    buf, norm = torch.ones(100, device=DEV), torch.empty(1, device=DEV)
    for grads, outs in (([buf, buf], None), ([buf[:60], buf[59:]], None), ([buf[50:], buf[:51]], None),
                        ([buf[:50]], [buf[1:51]]), ([buf[:50], buf[50:]], [buf[50:], buf[:50]])):
        with pytest.raises(la.KfacError):
            la.kfac_grad_clip(grads, 0.5, norm, outs=outs)
    torch.cuda.synchronize()
    assert bool((buf == 1).all())
    la.kfac_grad_norm([buf, buf], norm)       # the norm alone only reads
    assert abs(float(norm) - math.sqrt(200)) <= 2.0 ** -20


def test_memory_around_stays():
    """Elements next to the gradients keep their values."""
    import torch
    buf = torch.full((40001,), 2.0, device=DEV)
    low = torch.full((20003,), 2.0, device=DEV, dtype=torch.bfloat16)
    norm = torch.empty(1, device=DEV)
    la.kfac_grad_clip([buf[1:9000], buf[9001:40000], low[3:20000]], 1.0, norm)
    assert bool((buf[[0, 9000, 40000]] == 2).all()) and bool((low[:3] == 2).all()) and bool((low[20000:] == 2).all())
    assert bool((buf[1:9000] < 0.1).all()) and bool((low[3:20000] < 0.1).all())


def test_captured_and_on_another_stream():
    import torch
    sizes = [70000, 3, 9001, 0, 555] * 40
    base = gradients(sizes, ("f32", "bf16"))
    outs, norm = [torch.empty_like(t) for t in base], torch.empty(1, device=DEV)

    def step(stream=None):
        la.kfac_grad_clip(base, 2.0, norm, outs=outs, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        base[0].mul_(1.5)
        step()
        torch.cuda.synchronize()
        want, n = [t.clone() for t in outs], norm.clone()
        for run in (graph.replay, lambda: step(torch.cuda.Stream())):
            for t in (*outs, norm):
                t.fill_(-1.0)
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert torch.equal(n, norm) and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_a_tensor_of_more_than_32_bits():
    """Offsets past 2^32 elements; every block of 8 holds the same numbers, whose squares add up exactly."""
    import torch
    n, room = 2 ** 32 + 8, 64
    few = torch.tensor([1.0, -2.0, 3.0, 0.5, -0.25, 4.0, 0.0, 1.5], dtype=torch.bfloat16, device=DEV)
    big = torch.full((n + room,), 7.0, dtype=torch.bfloat16, device=DEV)
    big[:n].view(-1, 8).copy_(few)
    small = torch.ones(5, device=DEV)
    total = n // 8 * float(few.double().square().sum()) + 5
    norm = torch.empty(1, device=DEV)
    la.kfac_grad_clip([small, big[:n]], math.sqrt(total) / 2, norm)
    assert abs(float(norm) - math.sqrt(total)) <= 1.01 * ref.U32 * math.sqrt(total)
    # halves, but for the float32 norm and factor: a step of either, far less than one of bfloat16
    assert torch.equal(big[:n].view(-1, 8), (few / 2).expand(n // 8, 8)) and bool((big[n:] == 7.0).all())
    assert float((small - 0.5).abs().max()) <= 4 * ref.U32
