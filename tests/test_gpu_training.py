"""GPU: the differentiable attention, the layer that keeps its input, and both
under the preconditioner, against float64 autograd and the library's own calls."""
import os
import sys

import pytest

import linear_algebra_amd as la
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def plain_attention(q, k, v, bias, borders, lens):
    import torch
    n = q.shape[1]
    i = torch.arange(n, device=q.device)
    d = i - i[:, None]
    at = (d > 0) * (len(borders) + 1)
    for b in borders:
        at = at + (d.abs() >= b)
    s = torch.matmul(q.transpose(1, 2), k.transpose(1, 2).transpose(2, 3)) * q.shape[3] ** -0.5 + bias.t()[:, at]
    s = s.masked_fill(i >= lens[:, None, None, None], -float("inf"))
    return torch.matmul(torch.softmax(s, 3), v.transpose(1, 2)).transpose(1, 2)


def test_attention_autograd():
    """Gradients through views of one projection's output, float32, against
    float64 autograd: the softmax's sums have at most 150 terms of order one,
    and the dot products 32, so 2^-24 times a few hundred relative to the
    tensor's largest magnitude."""
    import torch
    from linear_algebra_amd.training import attention
    torch.manual_seed(0)
    borders = [1, 2, 5, 11]
    lens = torch.tensor([150, 77], dtype=torch.int32, device=DEV)
    x = torch.randn(2, 150, 3, 3, 32, device=DEV, requires_grad=True)
    bias = torch.randn(10, 3, device=DEV, requires_grad=True)
    w = torch.randn(2, 150, 3, 32, device=DEV)
    y = attention(x[:, :, 0], x[:, :, 1], x[:, :, 2], bias=bias, borders=borders, lens=lens)
    (y * w).sum().backward()
    xd, bd = x.detach().double().requires_grad_(), bias.detach().double().requires_grad_()
    yd = plain_attention(xd[:, :, 0], xd[:, :, 1], xd[:, :, 2], bd, borders, lens)
    (yd * w.double()).sum().backward()
    for name, got, want in (("y", y, yd), ("dx", x.grad, xd.grad), ("dbias", bias.grad, bd.grad)):
        err = float((got.double() - want).abs().max() / want.abs().max())
        say(f"  {name} {err:.2e}")
        assert err <= 512 * 2.0 ** -24


def test_kept_linear():
    """Output as torch.nn.Linear's; gradients those of the kept input."""
    import torch
    from linear_algebra_amd.training import CheckpointLinear
    torch.manual_seed(1)
    for bias in (True, False):
        m = CheckpointLinear(70, 33, bias=bias).to(DEV)
        x = torch.randn(4, 25, 70, device=DEV, requires_grad=True)
        w = torch.randn(4, 25, 33, device=DEV)
        y = m(x)
        assert torch.equal(y, torch.nn.functional.linear(x, m.weight, m.bias))
        y.backward(w)
        codes, scales, rows, batch = m.kept
        assert (rows, batch) == (100, 4)
        xh = torch.empty(100, 70, device=DEV)
        la.kfac_checkpoint_load([codes], [scales], [xh])
        # half a step of 3 + 1 bits, a third of the block's values at most one binade lower: under 2^-4 of the largest
        assert float((xh - x.detach().reshape(100, 70)).abs().max()) <= float(x.detach().abs().max()) * 2.0 ** -4
        g, xd = w.double().reshape(100, 33), xh.double()
        lim = 116 * 2.0 ** -24 * (g.abs().t() @ xd.abs())
        assert bool(((m.weight.grad.double() - g.t() @ xd).abs() <= 3 * lim).all())
        if bias:
            assert bool(((m.bias.grad.double() - g.sum(0)).abs() <= 3 * 116 * 2.0 ** -24 * g.abs().sum(0)).all())
        dx = (w.double().reshape(100, 33) @ m.weight.detach().double()).reshape(4, 25, 70)
        assert float((x.grad.double() - dx).abs().max()) <= 1e-5 * float(dx.abs().max())
        m.eval()
        before = m.kept
        m(x)
        assert m.kept is before


def test_kept_linear_bf16_input():
    import torch
    from linear_algebra_amd.training import CheckpointLinear
    m = CheckpointLinear(64, 32).to(DEV)
    x = torch.randn(3, 20, 64, device=DEV).bfloat16().requires_grad_()
    y = m(x)
    assert y.dtype == torch.bfloat16
    y.float().sum().backward()
    assert m.weight.grad.dtype == torch.float32 and x.grad.dtype == torch.bfloat16
    assert torch.equal(m.bias.grad, torch.full((32,), 60.0, device=DEV))


def test_preconditioner_takes_kept_inputs():
    """A model of kept and plain layers: every factor and preconditioned
    gradient as the library's calls give them on the layers' inputs."""
    import torch
    from linear_algebra_amd.kfac_preconditioner import KFACPreconditioner
    from linear_algebra_amd.training import CheckpointLinear
    torch.manual_seed(2)
    model = torch.nn.Sequential(CheckpointLinear(40, 50), torch.nn.ReLU(), torch.nn.Linear(50, 30), torch.nn.ReLU(),
                                CheckpointLinear(30, 7, bias=False)).to(DEV)
    pre = KFACPreconditioner(model, damping=1e-2, factor_decay=0.9, inv_update_freq=1)
    x = torch.randn(64, 40, device=DEV)
    first = True
    A = {}
    for _ in range(2):
        model.zero_grad()
        model(x + 0.1).square().mean().backward()
        grads = [m.weight.grad.clone() for m in (model[0], model[2], model[4])]
        pre.step()
        for k, m in enumerate((model[0], model[4])):
            codes, scales, rows, _ = m.kept
            f = A.setdefault(k, torch.zeros(codes.shape[1], codes.shape[1], device=DEV))
            la.kfac_checkpoint_factors([codes], [scales], [rows], [f], 0.9, first)
            assert torch.equal(torch.triu(pre.A[2 * k]), torch.triu(f))
        first = False
        for m, g in zip((model[0], model[2], model[4]), grads):
            assert torch.isfinite(m.weight.grad).all() and not torch.equal(m.weight.grad, g)
    assert pre.failed == []


def test_example_learns():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_encoder
    finally:
        sys.path.pop(0)
    losses = train_encoder.train(steps=40, say=lambda s: say(" ", s))
    assert sum(losses[-5:]) / 5 < 0.8 * sum(losses[:3]) / 3


@pytest.mark.parametrize("power", [1, 2])
def test_second_derivatives_are_refused(power):
    """What the kernels compute is not differentiated again: asking for it
    raises, also where the gradient that comes in is constant (power 1) and
    where another term of the sum has a graph, instead of dropping terms."""
    import torch
    from linear_algebra_amd.training import CheckpointLinear, attention
    torch.manual_seed(3)
    q, k, v = (torch.randn(1, 9, 2, 16, device=DEV, requires_grad=True) for _ in range(3))
    bias = torch.randn(4, 2, device=DEV, requires_grad=True)
    m = CheckpointLinear(16, 8).to(DEV)
    x = torch.randn(5, 16, device=DEV, requires_grad=True)
    for run, leaves, refused in ((lambda: attention(q, k, v, bias=bias, borders=[3]), (q, k, v, bias), (q, k, v, bias)),
                                 (lambda: m(x), (x, m.weight, m.bias), (m.weight, m.bias))):
        loss = run().pow(power).sum()
        grads = torch.autograd.grad(loss, refused, create_graph=True)
        for g in grads:
            for leaf in leaves:
                with pytest.raises(RuntimeError, match="second derivatives"):
                    torch.autograd.grad(run().sum() + g.square().sum(), leaf, retain_graph=True)
            with pytest.raises(RuntimeError, match="second derivatives"):
                (run().sum() + g.square().sum()).backward(retain_graph=True)


def test_second_derivative_of_the_kept_layers_input_gradient():
    """dx = gy W is torch's own product: a penalty on it gives the gradients that torch.nn.Linear gives."""
    import torch
    from linear_algebra_amd.training import CheckpointLinear
    torch.manual_seed(3)
    m, plain = CheckpointLinear(16, 8).to(DEV), torch.nn.Linear(16, 8).to(DEV)
    plain.load_state_dict(m.state_dict())
    x = torch.randn(5, 16, device=DEV, requires_grad=True)
    got = []
    for layer in (m, plain):
        dx, = torch.autograd.grad(layer(x).sum(), x, create_graph=True)
        got.append(torch.autograd.grad(dx.square().sum(), layer.weight)[0])
    assert torch.equal(*got)


def test_lengths_changed_before_the_backward_pass_are_noticed():
    import torch
    from linear_algebra_amd.training import attention
    q = torch.randn(2, 40, 2, 16, device=DEV, requires_grad=True)
    lens = torch.tensor([40, 7], dtype=torch.int32, device=DEV)
    y = attention(q, q, q, lens=lens)
    lens.fill_(40)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_borders_changed_before_the_backward_pass_change_nothing():
    import torch
    from linear_algebra_amd.training import attention
    torch.manual_seed(4)
    q = torch.randn(2, 40, 2, 16, device=DEV, requires_grad=True)
    bias = torch.randn(6, 2, device=DEV, requires_grad=True)
    for borders, other in (([2, 9], [5, 30]), (torch.tensor([2, 9]), torch.tensor([5, 30]))):
        got = []
        for change in (False, True):
            now = list(borders) if isinstance(borders, list) else borders.clone()
            y = attention(q, q, q, bias=bias, borders=now)
            if change:
                now[:] = other
            got.append(torch.autograd.grad(y.square().sum(), (q, bias)))
        for a, b in zip(*got):
            assert torch.equal(a, b)


def test_preconditioner_leaves_other_layers_attributes_alone():
    """A layer of the user's own with an attribute named like CheckpointLinear's is a plain layer."""
    import torch
    from linear_algebra_amd.kfac_preconditioner import KFACPreconditioner

    class Pruned(torch.nn.Linear):
        kept = 0.5                      # share of the weights kept

    grads = []
    for kind in (torch.nn.Linear, Pruned):
        torch.manual_seed(5)
        model = torch.nn.Sequential(kind(20, 12), torch.nn.ReLU(), kind(12, 5)).to(DEV)
        pre = KFACPreconditioner(model, damping=1e-2)
        model(torch.randn(32, 20, device=DEV)).square().mean().backward()
        assert all(t is not None for t in pre.factor_inputs()[0])
        pre.step()
        grads.append([p.grad for p in model.parameters()])
    for a, b in zip(*grads):
        assert torch.equal(a, b)


def test_workspaces_come_from_the_stream_that_uses_them(monkeypatch):
    """A block that torch's allocator hands out on one stream may still be in
    use by that stream's earlier work: the workspace of a call on another
    stream is taken on that other one."""
    import torch
    side = torch.cuda.Stream()
    seen, empty = [], torch.empty

    def noted(*a, **k):
        t = empty(*a, **k)
        if t.dtype == torch.uint8 and t.is_cuda:
            seen.append(torch.cuda.current_stream())
        return t

    q = torch.randn(2, 40, 4, 16, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(2, 4, 40, device=DEV)
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    bias = torch.zeros(6, 4, device=DEV)
    form = dict(bias=bias, borders=[3, 2000])
    x = torch.randn(4096, 33, device=DEV)
    codes, scales = la.kfac_checkpoint_empty(4096, 33, DEV)
    la.kfac_checkpoint_store([x], [codes], [scales])
    m, mat = torch.zeros(33, 33, device=DEV), torch.empty(33, 33, device=DEV)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", noted)
    for stream in (side, None):
        seen.clear()
        la.kfac_attention_forward(q, q, q, out, lse, stream=stream, **form)
        la.kfac_attention_backward(q, q, q, out, lse, q, dq, dk, dv, torch.empty_like(bias), stream=stream, **form)
        la.kfac_checkpoint_factors([codes], [scales], [4096], [m], 0.9, True, stream=stream)
        la.kfac_checkpoint_grad([x], [codes], [scales], [mat], stream=stream)
        la.kfac_factors([x], [m], 0.9, True, stream=stream)
        torch.cuda.synchronize()
        want = side if stream is not None else torch.cuda.current_stream()
        assert len(seen) == 5 and all(s == want for s in seen), (seen, want)


def test_kept_linear_without_rows():
    """An empty batch, as torch.nn.Linear takes it: empty output, gradients 0."""
    import torch
    from linear_algebra_amd.training import CheckpointLinear
    for bias in (True, False):
        m = CheckpointLinear(20, 6, bias=bias).to(DEV)
        for shape in ((0, 20), (3, 0, 20)):
            x = torch.empty(shape, device=DEV, requires_grad=True)
            m.zero_grad()
            y = m(x)
            assert y.shape == shape[:-1] + (6,)
            y.sum().backward()
            assert x.grad.shape == shape and not any(p.grad.any() for p in m.parameters())
            assert m.kept[2] == 0


def test_attention_takes_rows_that_lie_far_apart():
    """Rows further apart than the kernels' row stride limit are copied."""
    import torch
    from linear_algebra_amd.training import attention
    far = (1 << 30) // 128 // 4 + 4
    wide = torch.randn(2 * far + 32, device=DEV)
    q = wide.as_strided((1, 3, 2, 16), (0, far, 16, 1))
    assert torch.equal(attention(q, q, q), attention(*[q.contiguous()] * 3))
