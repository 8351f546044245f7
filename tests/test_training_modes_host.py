"""Layer norm and the gated block under torch's forward mode, functional
transforms and tracing, with plain operations in the kernels' place: a result
that these could not follow is refused, never wrong."""
import pytest

import linear_algebra_amd as la  # noqa: F401


@pytest.fixture
def stubs(monkeypatch):
    """The kernels' formulas on the host, written where the kernels would write."""
    import torch
    from linear_algebra_amd import training

    def norm(x, y, mean=None, rstd=None, weight=None, bias=None, eps=1e-5, stream=None):
        with torch.no_grad():
            m = x.detach().mean(1, keepdim=True)
            r = ((x.detach() - m).square().mean(1, keepdim=True) + eps).rsqrt()
            v = (x.detach() - m) * r * (1 if weight is None else weight.detach()) + (0 if bias is None else bias.detach())
            y.detach().data.copy_(v)
            if mean is not None:
                mean.copy_(m[:, 0]), rstd.copy_(r[:, 0])

    def gated(x, weight, h, bias=None, pre=None, activation="silu", stream=None):
        with torch.no_grad():
            p = x.detach() @ weight.detach().t() + (0 if bias is None else bias.detach())
            n = p.shape[1] // 2
            h.detach().data.copy_(torch.nn.functional.silu(p[:, :n]) * p[:, n:])
            if pre is not None:
                pre.copy_(p)

    monkeypatch.setattr(training, "kfac_layer_norm_forward", norm)
    monkeypatch.setattr(training, "kfac_gated_forward", gated)
    return training


def calls(training):
    import torch
    g = torch.Generator().manual_seed(1)
    w, b, wt = (torch.randn(s, generator=g) for s in ((6,), (6,), (10, 6)))
    return {"layer_norm": lambda x: training.layer_norm(x, w, b), "gated_linear": lambda x: training.gated_linear(x, wt)}


def plain(name, training, x):
    import torch
    g = torch.Generator().manual_seed(1)
    w, b, wt = (torch.randn(s, generator=g) for s in ((6,), (6,), (10, 6)))
    if name == "layer_norm":
        return torch.nn.functional.layer_norm(x, (6,), w, b)
    p = x @ wt.t()
    return torch.nn.functional.silu(p[..., :5]) * p[..., 5:]


NAMES = ["layer_norm", "gated_linear"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("grad", [False, True])
def test_values(stubs, name, grad):
    import torch
    x = torch.randn(2, 3, 6, requires_grad=grad)
    y = calls(stubs)[name](x)
    assert y.requires_grad == grad and torch.allclose(y.detach(), plain(name, stubs, x.detach()), atol=1e-5)
    with torch.no_grad():
        assert not calls(stubs)[name](x).requires_grad


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(stubs, name, grad):
    """A tangent that cannot be carried on raises; it is not dropped."""
    import torch
    import torch.autograd.forward_ad as fwd
    f, x, t = calls(stubs)[name], torch.randn(4, 6, requires_grad=grad), torch.randn(4, 6)
    with fwd.dual_level():
        with pytest.raises((RuntimeError, NotImplementedError)):
            f(fwd.make_dual(x, t))
        with torch.no_grad(), pytest.raises((RuntimeError, NotImplementedError)):
            f(fwd.make_dual(x.detach(), t))
        # a tangent of the weight alone, too
        w = fwd.make_dual(torch.ones(6), torch.randn(6))
        with pytest.raises((RuntimeError, NotImplementedError)):
            if name == "layer_norm":
                stubs.layer_norm(x, w)
            else:
                stubs.gated_linear(x, fwd.make_dual(torch.ones(10, 6), torch.randn(10, 6)))
        # without one, values as ever
        assert torch.allclose(f(x).detach(), plain(name, stubs, x.detach()), atol=1e-5)


@pytest.mark.parametrize("name", NAMES)
def test_functional_transforms_are_refused(stubs, name):
    import torch
    f = calls(stubs)[name]
    with pytest.raises(RuntimeError):
        torch.func.vmap(f)(torch.randn(5, 4, 6))
    with pytest.raises((RuntimeError, NotImplementedError)):
        torch.func.jvp(f, (torch.randn(4, 6),), (torch.randn(4, 6),))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kind", ["function", "module"])
def test_traced_programs_compute(stubs, name, kind):
    """A traced pass, gradients off, gives the values of its own inputs, not of
    memory that nothing in it writes."""
    import torch
    g = torch.Generator().manual_seed(2)
    a, b = torch.randn(4, 6, generator=g), torch.randn(4, 6, generator=g)
    if kind == "function":
        f = calls(stubs)[name]
    else:
        torch.manual_seed(3)
        f = stubs.LayerNorm(6).eval() if name == "layer_norm" else stubs.GatedLinear(6, 5).eval()
    with torch.no_grad():
        traced = torch.jit.trace(f, (a,), check_trace=False)
        for x in (a, b, a):
            got = traced(x)
            torch.empty(4, 5).fill_(77.0)
            assert torch.equal(got, f(x))


@pytest.mark.parametrize("name", NAMES)
def test_inference_mode(stubs, name):
    import torch
    x = torch.randn(4, 6)
    with torch.inference_mode():
        y = calls(stubs)[name](x)
    assert y.is_inference() and torch.allclose(y.clone(), plain(name, stubs, x), atol=1e-5)


def test_layers_kept_without_the_choice_of_rounding(stubs):
    """A layer that was stored before it had that choice rounds."""
    import torch
    layer = stubs.GatedLinear(6, 5)
    layer.__dict__.pop("unrounded", None)
    assert layer(torch.randn(4, 6)).shape == (4, 5)
