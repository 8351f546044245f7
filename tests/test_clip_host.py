"""Host side of clip_grad_norm_: what it refuses, by name, and what it takes
for the largest norm (nothing reaches the GPU)."""
import os
import re

import pytest

import linear_algebra_amd as la

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def parameters(n):
    import torch
    flat = torch.zeros(n)
    got = []
    for k in range(n):
        p = torch.nn.Parameter(torch.zeros(1))
        p.grad = flat[k:k + 1]
        got.append(p)
    return got


def test_too_many_gradients_are_named():
    """4096 get as far as the device, one more is refused with the limit."""
    import torch
    from linear_algebra_amd import training
    many = parameters(4097)
    with pytest.raises(ValueError, match="4097 gradients.* at most 4096"):
        training.clip_grad_norm_(many, 1.0)
    with pytest.raises(ValueError, match="GPU"):
        training.clip_grad_norm_(many[:4096], 1.0)
    with pytest.raises(ValueError, match="at most 4096"):
        la.kfac_grad_norm([p.grad for p in many], torch.zeros(1))
    with pytest.raises(ValueError, match="at most 4096"):
        la.kfac_grad_clip([p.grad for p in many], 1.0, torch.zeros(1))
    # the limit is the library's
    header = open(os.path.join(ROOT, "include", "kfac.h")).read()
    assert int(re.search(r"#define KFAC_MAX_COUNT (\d+)", header).group(1)) == la.KFAC_MAX_COUNT


@pytest.mark.parametrize("kind", ["int", "numpy", "tensor"])
def test_the_largest_norm_may_be_any_number(monkeypatch, kind):
    import numpy
    import torch
    from linear_algebra_amd import training
    seen = []
    monkeypatch.setattr(training, "kfac_grad_clip", lambda grads, most, norm: seen.append(most))
    p = torch.nn.Parameter(torch.zeros(3))
    p.grad = torch.ones(3)
    training.clip_grad_norm_(p, {"int": 2, "numpy": numpy.float32(2.0), "tensor": torch.tensor(2.0)}[kind])
    assert type(seen[0]) is float and seen[0] == 2.0
