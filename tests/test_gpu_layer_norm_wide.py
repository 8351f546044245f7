"""GPU: layer norm of the widest rows, with more of them than the card takes at
once, so that every form goes from row to row; and with integers, whose sums
over many rows are exact."""
import pytest

import linear_algebra_amd as la
from tests import encoder_reference as ref
from tests.gpu_helpers import DEV, say
from tests.test_gpu_layer_norm import FORMS, forward, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,weight_dtype", FORMS)
@pytest.mark.parametrize("rows,d", [(300, 8193), (700, 9217), (523, 12345), (257, 16384), (1100, 6145), (900, 8192)])
def test_more_rows_than_workgroups(rows, d, dtype, weight_dtype):
    import torch
    x, dy, w, b = inputs(rows, d, dtype, weight_dtype)
    y, mean, rstd = forward(x, w, b)
    want = ref.norm_forward(x, w, b, 1e-5, dtype)
    got = {"y": y, "mean": mean, "rstd": rstd}
    dx = torch.full((rows, d), float("nan"), dtype=x.dtype, device=DEV)
    dw, db = (torch.full((d,), float("nan"), dtype=w.dtype, device=DEV) for _ in range(2))
    la.kfac_layer_norm_backward(dy.to(DEV), x.to(DEV), mean, rstd, dx, weight=w.to(DEV), dweight=dw, dbias=db)
    want.update(ref.norm_backward(dy, x, mean.cpu(), rstd.cpu(), w, dtype, weight_dtype))
    got.update(dx=dx, dweight=dw, dbias=db)
    for name, value in got.items():
        r = ref.worst(value, *want[name])
        say(f"  {name} {r:.3f}")
        assert r <= 1.0, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,d", [(1, 3), (5, 8), (4099, 40), (20001, 64), (3001, 200), (2001, 1000), (1500, 1025), (4001, 2304),
                                    (700, 5000), (523, 12345)])
def test_sums_over_rows_are_exact_on_integers(rows, d, dtype):
    """Statistics 0 and 1 make xh = x: dweight and dbias are sums of integers,
    so that a row lost or taken twice shows at any number of rows."""
    import torch
    g = torch.Generator(device=DEV).manual_seed(rows + d)
    x, dy = (torch.randint(-2, 3, (rows, d), generator=g, device=DEV).to(ref.types()[dtype]) for _ in range(2))
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    dw, db = (torch.full((d,), float("nan"), device=DEV) for _ in range(2))
    la.kfac_layer_norm_backward(dy, x, mean, rstd, dweight=dw, dbias=db)
    assert torch.equal(dw.double(), (dy.double() * x.double()).sum(0)) and torch.equal(db.double(), dy.double().sum(0))
