"""GPU: the gated block where the parts of float32 operands, and float32 dpre
beside bfloat16 rows, lie past 32 bits of offset.  Integers: every output is exact."""
import pytest

import linear_algebra_amd as la
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu

ROWS = 2 ** 28 + 13     # a plane of parts holds 8 numbers of each row


@pytest.mark.parametrize("dtype", ["f32", "mixed"])
def test_backward(dtype):
    import torch
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-2, 3, (8, 2), generator=g, device=DEV).to(t).repeat(ROWS // 8 + 1, 1)[:ROWS].contiguous()
    w = torch.tensor([[1.0, -2.0], [3.0, 1.0]], device=DEV).to(t)
    # gradients in the first and the last rows and in some between: sums that stay small
    dh = torch.zeros(ROWS, 1, dtype=t, device=DEV)
    at = torch.tensor([0, 1, 127, 128, 2 ** 27 - 1, 2 ** 27, 2 ** 28 - 1, 2 ** 28, 2 ** 28 + 4, ROWS - 2, ROWS - 1], device=DEV)
    dh[at, 0] = torch.arange(1, len(at) + 1, device=DEV).to(t)
    pre = torch.ones(ROWS, 2, dtype=t, device=DEV)
    dpre = torch.full((ROWS + 8, 2), 7.0, device=DEV)
    dx = torch.full((ROWS + 8, 2), 7.0, dtype=t, device=DEV)
    dw, db = torch.empty(2, 2, device=DEV), torch.empty(2, device=DEV)
    la.kfac_gated_backward(dh, x, w, pre, dpre[:ROWS], dx[:ROWS], dw, db, activation="relu")
    for k in range(2):
        assert torch.equal(dpre[:ROWS, k], dh[:, 0].float())
        assert torch.equal(dx[:ROWS, k], dh[:, 0] * (w[0, k] + w[1, k]))
    assert bool((dpre[ROWS:] == 7).all()) and bool((dx[ROWS:] == 7).all())
    few = (dh[at].double() * x[at].double()).sum(0)
    assert torch.equal(dw.double(), few.expand(2, 2)) and torch.equal(db.double(), dh[at].double().sum().expand(2))


def test_forward_float32():
    import torch
    few = torch.tensor([[1.0, 2.0], [-1.0, 3.0], [2.0, 0.0], [0.5, -4.0]], device=DEV)
    x = few.repeat(ROWS // 4 + 1, 1)[:ROWS].contiguous()
    w = torch.tensor([[1.0, -2.0], [3.0, 1.0]], device=DEV)
    pre, h = torch.full((ROWS + 8, 2), 7.0, device=DEV), torch.full((ROWS + 8, 1), 7.0, device=DEV)
    la.kfac_gated_forward(x, w, h[:ROWS], pre=pre[:ROWS], activation="relu")
    p = few @ w.t()
    want = (p[:, 0].clamp_min(0) * p[:, 1])[:, None]
    whole = ROWS // 4 * 4
    assert torch.equal(pre[:whole].view(-1, 4, 2), p.expand(whole // 4, 4, 2)) and torch.equal(pre[whole:ROWS], p[:ROWS - whole])
    assert torch.equal(h[:whole].view(-1, 4, 1), want.expand(whole // 4, 4, 1)) and torch.equal(h[whole:ROWS], want[:ROWS - whole])
    assert bool((pre[ROWS:] == 7).all()) and bool((h[ROWS:] == 7).all())
