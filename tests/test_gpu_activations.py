"""GPU: the gated block's activations and their slopes in float32, each to its
own relative precision far into its tail."""
import math

import pytest

import linear_algebra_amd as la
from tests.gpu_helpers import DEV, say
from tests.encoder_reference import U32

pytestmark = pytest.mark.gpu

# Bounds in half steps of float32, for exp2 and the reciprocal within a step
# (two halves) each.  Of the logistic function: exp2 2, the first-order term 1,
# 1 + e 1, the reciprocal 2, their product 1.  Of the normal tail: its
# exponential 4 (two more products), the polynomial's ten steps and its argument
# 7, their product 1.  An activation has one more product.  A slope q (1 + g p),
# q p, q + g phi or q + g q p c (1 + 0.13 g^2) adds up its factors' and its own
# roundings, in parts of the sum of its terms' magnitudes.  A tenth for second orders.
STEPS = {"silu": (8, 18), "sigmoid": (7, 15), "gelu": (13, 16), "gelu_tanh": (8, 24)}
FAR = {"silu": 86.0, "sigmoid": 86.0, "gelu": 12.8, "gelu_tanh": 10.0}


def exact(act, g):
    """(act, slope, the sum of the slope's terms' magnitudes), float64."""
    import torch
    if act in ("silu", "sigmoid"):
        q, p = torch.sigmoid(g), torch.sigmoid(-g)
        return (q, q * p, q * p) if act == "sigmoid" else (g * q, q * (1 + g * p), q * (1 + g.abs() * p))
    if act == "gelu":
        q, t = 0.5 * torch.erfc(-g / math.sqrt(2)), g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        c = math.sqrt(8 / math.pi)
        z = c * (g + 0.044715 * g ** 3)
        q, p = torch.sigmoid(z), torch.sigmoid(-z)
        t = g * q * p * c * (1 + 0.134145 * g * g)
    return g * q, q + t, q + t.abs()


def gates(act):
    import torch
    far = FAR[act]
    r = torch.Generator().manual_seed(7)
    return torch.cat([torch.linspace(-far, far, 9000), (torch.rand(5000, generator=r) - 0.5) * 6, torch.logspace(-30, 0, 300),
                      -torch.logspace(-30, 0, 300)])


@pytest.mark.parametrize("act", list(STEPS))
def test_relative_precision(act):
    import torch
    g = gates(act)
    n = g.numel()
    a, slope, size = exact(act, g.double())
    x, w = torch.zeros(1, 8, device=DEV), torch.zeros(2 * n, 8, device=DEV)
    pre, ones = torch.cat([g, torch.ones(n)])[None].to(DEV), torch.ones(1, n, device=DEV)
    h, dpre = torch.empty(1, n, device=DEV), torch.empty(1, 2 * n, device=DEV)
    la.kfac_gated_forward(x, w, h, bias=pre[0], activation=act)
    la.kfac_gated_backward(ones, x, w, pre, dpre, activation=act)
    small = 2.0 ** -126 * U32 * 8                     # where a factor leaves the normal numbers
    for name, got, want, scale, steps in (("h", h[0], a, a.abs(), STEPS[act][0]), ("du", dpre[0, n:], a, a.abs(), STEPS[act][0]),
                                          ("dg", dpre[0, :n], slope, size, STEPS[act][1])):
        r = float(((got.double().cpu() - want).abs() / (1.1 * steps * U32 * scale + small)).max())
        say(f"  {act} {name} {r:.3f} of {steps} half steps")
        assert r <= 1.0, name


@pytest.mark.parametrize("act", list(STEPS))
def test_far_out_and_no_numbers(act):
    """Past the bend: 0, the gate itself or 1, and slopes 0 and 1; infinities
    do not become NaN where the formula has a value; NaN stays NaN."""
    import torch
    inf = float("inf")
    g = torch.tensor([150.0, 300.0, 3e4, 1e19, 1e38, 3.4e38, inf, -150.0, -300.0, -3e4, -1e19, -1e38, -3.4e38, float("nan")])
    n = g.numel()
    x, w = torch.zeros(1, 8, device=DEV), torch.zeros(2 * n, 8, device=DEV)
    pre, ones = torch.cat([g, torch.ones(n)])[None].to(DEV), torch.ones(1, n, device=DEV)
    h, dpre = torch.empty(1, n, device=DEV), torch.empty(1, 2 * n, device=DEV)
    la.kfac_gated_forward(x, w, h, bias=pre[0], activation=act)
    la.kfac_gated_backward(ones, x, w, pre, dpre, activation=act)
    h, dg, du = h[0].cpu(), dpre[0, :n].cpu(), dpre[0, n:].cpu()
    top = torch.ones(7) if act == "sigmoid" else g[:7]
    assert torch.equal(h[:7], top) and torch.equal(du[:7], top)
    assert not h[7:13].any() and not du[7:13].any()
    assert torch.equal(dg[:6], torch.zeros(6) if act == "sigmoid" else torch.ones(6)) and not dg[7:13].any()
    assert bool(h[13].isnan()) and bool(du[13].isnan()) and bool(dg[13].isnan())
