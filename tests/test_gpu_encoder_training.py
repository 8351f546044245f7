"""GPU: layer norm, the gated block and clipping as a training program uses
them: under autograd, with attention in one layer, under the preconditioner,
in a captured graph."""
import math

import pytest

import linear_algebra_amd as la
from tests import encoder_reference as ref
from tests.gpu_helpers import DEV, say

pytestmark = pytest.mark.gpu


def layer(width, heads, inner, act, kind):
    """An encoder layer of this package (kind 'own') or of plain torch operations."""
    import torch
    from linear_algebra_amd import training

    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.norm1 = (training.LayerNorm if kind == "own" else torch.nn.LayerNorm)(width)
            self.norm2 = (training.LayerNorm if kind == "own" else torch.nn.LayerNorm)(width)
            self.qkv, self.out = torch.nn.Linear(width, 3 * width), torch.nn.Linear(width, width)
            self.up = training.GatedLinear(width, inner, activation=act) if kind == "own" else torch.nn.Linear(width, 2 * inner)
            self.down = torch.nn.Linear(inner, width)

        def forward(self, x, lens):
            b, n, _ = x.shape
            q, k, v = self.qkv(self.norm1(x)).view(b, n, 3, heads, width // heads).unbind(2)
            if kind == "own":
                y = training.attention(q, k, v, lens=lens)
            else:
                s = torch.matmul(q.transpose(1, 2), k.transpose(1, 2).transpose(2, 3)) * (width // heads) ** -0.5
                s = s.masked_fill(torch.arange(n, device=x.device) >= lens[:, None, None, None], -float("inf"))
                y = torch.matmul(torch.softmax(s, 3), v.transpose(1, 2)).transpose(1, 2)
            x = x + self.out(y.reshape(b, n, width))
            z = self.up(self.norm2(x))
            if kind != "own":
                z = ref.activation(act, z[..., :inner])[0] * z[..., inner:]
            return x + self.down(z)

    return Layer()


@pytest.mark.parametrize("act", list(la.KFAC_ACTIVATIONS))
def test_encoder_layer(act):
    """Output and every gradient against float64: ten sums behind one another,
    each of at most 256 terms of either sign, rounded in float32; sums of
    terms that cancel to a tenth of their size still leave 10 * 256 * 1.6 of
    2^-24 of the largest magnitude as a bound."""
    import torch
    torch.manual_seed(0)
    own = layer(64, 4, 90, act, "own").to(DEV)
    plain = layer(64, 4, 90, act, "plain").to(DEV).double()
    plain.load_state_dict({k: v.double() for k, v in own.state_dict().items()})
    x = torch.randn(2, 37, 64, device=DEV, requires_grad=True)
    w = torch.randn(2, 37, 64, device=DEV)
    lens = torch.tensor([37, 20], dtype=torch.int32, device=DEV)
    xd = x.detach().double().requires_grad_()
    y, yd = own(x, lens), plain(xd, lens)
    (y * w).sum().backward()
    (yd * w.double()).sum().backward()
    pairs = [("y", y, yd), ("x", x.grad, xd.grad)]
    pairs += [(n, p.grad, dict(plain.named_parameters())[n].grad) for n, p in own.named_parameters()]
    for name, got, want in pairs:
        err = float((got.double() - want).abs().max() / want.abs().max())
        say(f"  {name} {err:.2e}")
        assert err <= 4096 * ref.U32, name


@pytest.mark.parametrize("weight_type", ["f32", "bf16"])
def test_bf16_input(weight_type):
    """Outputs and gradients keep their tensors' types and shapes; the
    gradients are those of the library's calls."""
    import torch
    from linear_algebra_amd.training import GatedLinear, LayerNorm
    torch.manual_seed(1)
    t = ref.types()[weight_type]
    norm, up = LayerNorm((3, 20)).to(DEV).to(t), GatedLinear(20, 33, activation="relu").to(DEV).to(t)
    x = torch.randn(5, 3, 20, device=DEV).bfloat16().requires_grad_()
    a = norm(x)
    h = up(a)
    assert a.dtype == h.dtype == torch.bfloat16 and h.shape == (5, 3, 33)
    dh = torch.randn(5, 3, 33, device=DEV).bfloat16()
    h.backward(dh)
    assert x.grad.dtype == torch.bfloat16 and x.grad.shape == x.shape
    for p in (*norm.parameters(), *up.parameters()):
        assert p.grad.dtype == t and p.grad.shape == p.shape
    pre, out = torch.empty(15, 66, device=DEV).bfloat16(), torch.empty(15, 33, device=DEV).bfloat16()
    w, b = up.weight.detach().bfloat16(), up.bias.detach().float()
    la.kfac_gated_forward(a.detach().view(15, 20), w, out, bias=b, pre=pre, activation="relu")
    assert torch.equal(out.view(5, 3, 33), h)
    dpre, dx, dw, db = torch.empty_like(pre), torch.empty(15, 20, device=DEV).bfloat16(), torch.empty(66, 20, device=DEV), torch.empty_like(b)
    la.kfac_gated_backward(dh.view(15, 33), a.detach().view(15, 20), w, pre, dpre, dx, dw, db, activation="relu")
    assert torch.equal(up.weight.grad, dw.to(t)) and torch.equal(up.bias.grad, db.to(t))


def test_views_and_empty_batches():
    """Inputs that are views, expanded or transposed, and batches without rows."""
    import torch
    from linear_algebra_amd.training import gated_linear, layer_norm
    torch.manual_seed(2)
    base = torch.randn(6, 50, 41, device=DEV)
    w, wt = torch.randn(20, device=DEV), torch.randn(10, 20, device=DEV)
    views = [base[:, 3, 1:21], base[:, :, :20], base[:3, ::2, 5:25], base.transpose(1, 2)[:, :, :20],
             base[0, 0, :20].expand(4, 20), base[1, 2, :20]]
    for v in views:
        for f in (lambda t: layer_norm(t, w, w), lambda t: gated_linear(t, wt)):
            a, b = v.detach().requires_grad_(), v.detach().clone(memory_format=torch.contiguous_format).requires_grad_()
            ya, yb = f(a), f(b)
            assert torch.equal(ya, yb) and torch.equal(f(a.detach()), ya)
            # an expanded gradient too
            ya.sum().backward()
            yb.sum().backward()
            assert torch.equal(a.grad, b.grad)
    for shape in ((0, 20), (3, 0, 20)):
        x = torch.empty(shape, device=DEV, requires_grad=True)
        wp, gp = w.clone().requires_grad_(), wt.clone().requires_grad_()
        (layer_norm(x, wp).sum() + gated_linear(x, gp).sum()).backward()
        assert x.grad.shape == shape and not wp.grad.any() and not gp.grad.any()


def test_frozen_parts():
    """Only what asks for a gradient gets one, of the same bits."""
    import torch
    from linear_algebra_amd.training import gated_linear, layer_norm
    torch.manual_seed(3)
    for f, shapes in ((lambda x, w, b: layer_norm(x, w, b), ((40, 24), (24,), (24,))),
                      (lambda x, w, b: gated_linear(x, w, b, "gelu"), ((40, 24), (60, 24), (60,)))):
        full = [torch.randn(s, device=DEV, requires_grad=True) for s in shapes]
        want = torch.autograd.grad(f(*full).square().sum(), full)
        for keep in range(3):
            some = [t.detach().requires_grad_(k == keep) for k, t in enumerate(full)]
            got, = torch.autograd.grad(f(*some).square().sum(), some[keep])
            assert torch.equal(got, want[keep])
        with torch.no_grad():
            assert f(*full).grad_fn is None


def test_second_derivatives_are_refused():
    import torch
    from linear_algebra_amd.training import gated_linear, layer_norm
    torch.manual_seed(4)
    x, w, b = (torch.randn(s, device=DEV, requires_grad=True) for s in ((7, 16), (16,), (16,)))
    wt = torch.randn(12, 16, device=DEV, requires_grad=True)
    for run, leaves in ((lambda: layer_norm(x, w, b), (x, w)), (lambda: gated_linear(x, wt), (x, wt))):
        grads = torch.autograd.grad(run().square().sum(), leaves, create_graph=True)
        for g in grads:
            for leaf in leaves:
                with pytest.raises(RuntimeError, match="second derivatives"):
                    torch.autograd.grad(g.square().sum(), leaf, retain_graph=True)


def test_preconditioner_takes_the_gated_layer():
    """Factors and preconditioned gradients of a gated layer as the library's
    calls give them on its input and its projections' gradient."""
    import torch
    from linear_algebra_amd.kfac_preconditioner import KFACPreconditioner
    from linear_algebra_amd.training import CheckpointLinear, GatedLinear, LayerNorm
    torch.manual_seed(5)
    model = torch.nn.Sequential(torch.nn.Linear(30, 24), LayerNorm(24), GatedLinear(24, 20), CheckpointLinear(20, 5)).to(DEV)
    pre = KFACPreconditioner(model, damping=1e-2, factor_decay=0.9, inv_update_freq=1)
    seen = []
    model[2].output_grad_hooks.append(lambda m, g: seen.append(g))
    A, G = torch.zeros(25, 25, device=DEV), torch.zeros(40, 40, device=DEV)
    for step in range(2):
        model.zero_grad()
        x = torch.randn(64, 30, device=DEV)
        model(x).square().mean().backward()
        up = model[2]
        with torch.no_grad():
            inner = model[1](model[0](x))
        z = torch.nn.functional.linear(inner.double(), up.weight.double(), up.bias.double())
        h = torch.nn.functional.silu(z[:, :20]) * z[:, 20:]
        assert float((up(inner).double() - h).abs().max()) <= 1e-5 * float(h.abs().max())
        wg, bg = up.weight.grad.clone(), up.bias.grad.clone()
        pre.step()
        ones = torch.cat([inner, torch.ones(64, 1, device=DEV)], 1)
        la.kfac_factors([ones], [A], 0.9, step == 0)
        la.kfac_factors([seen[-1] * 64.0], [G], 0.9, step == 0)
        at = pre.layers.index(up)
        for got, want in ((pre.A[at], A), (pre.G[at], G)):
            assert torch.equal(torch.triu(got), torch.triu(want))
        out = torch.empty(40, 25, device=DEV)
        la.kfac_precondition([pre.Ginv[at]], [torch.cat([wg, bg[:, None]], 1)], [pre.Ainv[at]], [out])
        assert torch.equal(up.weight.grad, out[:, :24]) and torch.equal(up.bias.grad, out[:, 24])
    pre.remove()
    assert len(model[2].output_grad_hooks) == 1
    model[2].eval()
    model(x).sum().backward()
    assert len(seen) == 3


def test_clip_grad_norm():
    """The norm that torch's function gives, and its gradients, to float32's
    rounding (its norm is summed in float32: n additions of a tensor's squares)."""
    import torch
    from linear_algebra_amd.training import clip_grad_norm_
    torch.manual_seed(6)
    shapes = [(30, 40), (7,), (), (0, 3), (5, 6, 7, 8), (64, 3)]
    for max_norm in (0.5, 1e6):
        params = [torch.nn.Parameter(torch.zeros(s, device=DEV)) for s in shapes]
        for p in params:
            p.grad = torch.randn(p.shape, device=DEV)
        params[4].grad = torch.randn(8, 7, 6, 5, device=DEV).permute(3, 2, 1, 0)       # other orders of the same memory
        params[5].grad = torch.randn(64, 5, device=DEV)[:, :3]                         # and rows that lie apart
        params.append(torch.nn.Parameter(torch.zeros(3, device=DEV)))                  # no gradient
        before = [None if p.grad is None else p.grad.clone() for p in params]
        versions = [p.grad._version for p in params[:-1]]
        norm = clip_grad_norm_(iter(params), max_norm)
        want = math.sqrt(sum(float(g.double().square().sum()) for g in before if g is not None))
        assert norm.shape == () and abs(float(norm) - want) <= 1.01 * ref.U32 * want
        c = min(1.0, max_norm / (want + 1e-6))
        for p, g in zip(params, before):
            if g is not None:
                assert bool(((p.grad.double() - g.double() * c).abs() <= 3.02 * ref.U32 * g.double().abs()).all())
        assert all(p.grad._version > v for p, v in zip(params[:-1], versions))
    one = torch.nn.Parameter(torch.zeros(4, device=DEV))
    one.grad = torch.full((4,), 3.0, device=DEV)
    assert float(clip_grad_norm_(one, 1.0)) == 6.0
    shared = torch.nn.Parameter(torch.zeros(4, device=DEV))
    shared.grad = one.grad
    with pytest.raises(la.KfacError):
        clip_grad_norm_([one, shared], 1.0)


def test_training_step_in_a_graph():
    """Forward, backward and clipping of a layer, captured once and replayed on
    new inputs, give the eager step's bits."""
    import torch
    from linear_algebra_amd.training import GatedLinear, LayerNorm, clip_grad_norm_
    torch.manual_seed(7)
    model = torch.nn.Sequential(LayerNorm(96), GatedLinear(96, 130, activation="gelu")).to(DEV)
    x, w = torch.randn(200, 96, device=DEV), torch.randn(200, 130, device=DEV)
    params = list(model.parameters())
    for p in params:
        p.grad = torch.zeros_like(p)

    def step():
        for p in params:
            p.grad.zero_()
        (model(x) * w).sum().backward()
        return clip_grad_norm_(params, 1.0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    for _ in range(3):
        x.copy_(torch.randn(200, 96, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [norm.clone()] + [p.grad.clone() for p in params]
        want = [step().clone()] + [p.grad.clone() for p in params]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
