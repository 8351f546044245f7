"""GPU: the gated block on numbers whose sums are exact in float32 in any
order, so that a term lost, counted twice or put elsewhere, or a product of
parts left out, shows as a difference at any length of the reduction."""
import pytest

import linear_algebra_amd as la
from tests.gpu_helpers import DEV
from tests.test_gpu_gated import SHAPES
from tests.test_gpu_gated_large import BF16, F32

pytestmark = pytest.mark.gpu

CASES = [("bf16", *s) for s in SHAPES + BF16] + [("f32", *s) for s in SHAPES + F32]


def types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}


def draw(seed):
    import torch
    g = torch.Generator(device=DEV).manual_seed(seed)

    def ints(low, high, *shape, dtype):
        return torch.randint(low, high + 1, shape, generator=g, device=DEV).to(dtype)

    return g, ints


def nan(like, dtype=None):
    import torch
    return torch.full(like, float("nan"), dtype=dtype, device=DEV)


def same(got, want, name):
    """Equal to a float64 value that float32 holds, rounded once to the result's type."""
    import torch
    assert float(want.abs().max()) < 2 ** 24 if want.numel() else True
    assert torch.equal(want.float().double(), want), name
    assert torch.equal(got, want.float().to(got.dtype)), name


@pytest.mark.parametrize("dtype,rows,d,width", CASES)
def test_forward(dtype, rows, d, width):
    import torch
    t = types()[dtype]
    _, ints = draw(rows + 3 * d + 5 * width)
    x, w, b = ints(-1, 1, rows, d, dtype=t), ints(-1, 1, 2 * width, d, dtype=t), ints(-3, 3, 2 * width, dtype=torch.float32)
    h, pre = nan((rows, width), t), nan((rows, 2 * width), t)
    la.kfac_gated_forward(x, w, h, bias=b, pre=pre, activation="relu")
    want = x.double() @ w.double().t() + b.double()
    same(pre, want, "pre")
    same(h, want[:, :width].clamp_min(0) * want[:, width:], "h")


@pytest.mark.parametrize("dtype,rows,d,width", CASES + [("mixed", *s) for s in SHAPES + BF16])
def test_backward(dtype, rows, d, width):
    """mixed: bfloat16 rows with a float32 dpre."""
    import torch
    t = types().get(dtype, torch.bfloat16)
    _, ints = draw(rows + 5 * d + 3 * width)
    dh, x, w = ints(-1, 1, rows, width, dtype=t), ints(-1, 1, rows, d, dtype=t), ints(-1, 1, 2 * width, d, dtype=t)
    pre = ints(-1, 2, rows, 2 * width, dtype=t)
    got = {"dpre": nan((rows, 2 * width), torch.float32 if dtype == "mixed" else t), "dx": nan((rows, d), t),
           "dweight": nan((2 * width, d), torch.float32), "dbias": nan((2 * width,), torch.float32)}
    la.kfac_gated_backward(dh, x, w, pre, activation="relu", **got)
    g, u = pre[:, :width].double(), pre[:, width:].double()
    dpre = torch.cat([dh.double() * u * (g > 0), dh.double() * g.clamp_min(0)], 1)
    want = {"dpre": dpre, "dx": dpre @ w.double(), "dweight": dpre.t() @ x.double(), "dbias": dpre.sum(0)}
    for name in got:
        same(got[name], want[name], name)
    # each product by itself, which may share its tiles out otherwise
    for name in ("dx", "dweight"):
        one = torch.full_like(got[name], float("nan"))
        la.kfac_gated_backward(dh, x, w, pre, got["dpre"], activation="relu", **{name: one})
        same(one, want[name], name)


# ------------------------------------------------------------------- parts --

def parts(ints, count, *shape):
    """n0 + n1 2^-9 (+ n2 2^-18), each n -1, 0 or 1: as many bfloat16 parts,
    and sums of up to 15 of them fit float32's 24 bits."""
    import torch
    v = sum(ints(-1, 1, *shape, dtype=torch.float32) * 2.0 ** (-9 * k) for k in range(count))
    return v.contiguous()


def sparse(values, along):
    """At most 15 of the numbers left in each line of that dimension: the
    lines' stretches of a random order of its places, which they cover in turn."""
    import torch
    n, lines = values.shape[along], values.shape[1 - along]
    g = torch.Generator().manual_seed(n + lines)
    order = torch.randperm(n, generator=g)
    at = (torch.arange(lines)[:, None] * 15 + torch.arange(min(15, n))) % n
    mask = torch.zeros(lines, n)
    mask.scatter_(1, order[at], 1.0)
    mask = mask.to(DEV)
    return (values * (mask.t() if along == 0 else mask)).contiguous()


PARTS = [(200, 40, 50), (4100, 77, 45), (1834, 1445, 331), (1301, 515, 1203), (300, 16384, 40), (20001, 33, 9), (5000, 200, 300)]


@pytest.mark.parametrize("rows,d,width", PARTS)
def test_forward_takes_every_product_of_parts(rows, d, width):
    import torch
    _, ints = draw(rows + d)
    signs = [ints(0, 1, *s, dtype=torch.float32) * 2 - 1 for s in ((rows, d), (2 * width, d))]
    for nx, nw in ((3, 1), (1, 3), (2, 2)):
        x = parts(ints, nx, rows, d) if nx > 1 else sparse(signs[0], 1)
        w = sparse(parts(ints, nw, 2 * width, d) if nw > 1 else signs[1], 1) if nx > 1 else parts(ints, nw, 2 * width, d)
        h, pre = nan((rows, width), torch.float32), nan((rows, 2 * width), torch.float32)
        la.kfac_gated_forward(x, w, h, pre=pre, activation="relu")
        want = x.double() @ w.double().t()
        same(pre, want, (nx, nw))
        assert torch.equal(h, pre[:, :width].clamp_min(0) * pre[:, width:])


@pytest.mark.parametrize("dtype", ["f32", "mixed"])
@pytest.mark.parametrize("rows,d,width", PARTS)
def test_backward_takes_every_product_of_parts(rows, d, width, dtype):
    import torch
    t = types()["bf16" if dtype == "mixed" else "f32"]
    _, ints = draw(rows + d + 1)

    def signs(*shape):
        return ints(0, 1, *shape, dtype=torch.float32) * 2 - 1

    pre = signs(rows, 2 * width).to(t)
    g, u = pre[:, :width].double(), pre[:, width:].double()

    def run(dh, x, w, name):
        got = {"dpre": nan((rows, 2 * width), torch.float32), "dx": nan((rows, d), torch.float32 if dtype == "f32" else t),
               "dweight": nan((2 * width, d), torch.float32)}
        la.kfac_gated_backward(dh.to(t), x.to(t), w.to(t), pre, got["dpre"], activation="relu", **{k: got[k] for k in name})
        dpre = torch.cat([dh.double() * u * (g > 0), dh.double() * g.clamp_min(0)], 1)
        same(got["dpre"], dpre, "dpre")
        for k in name:
            same(got[k], dpre @ w.double() if k == "dx" else dpre.t() @ x.double(), (name, k))

    if dtype == "mixed":
        # dpre in two parts, from products of bfloat16 numbers
        dh = (signs(rows, width) * (1 + 2.0 ** -7)).bfloat16().float()
        pre[:, width:] = (signs(rows, width) * (1 + 2.0 ** -7)).to(t)
        u = pre[:, width:].double()
        # (1 + 2^-7)^2 = 1 + 2^-6 + 2^-14
        run(dh, sparse(signs(rows, d), 0), sparse(signs(2 * width, d), 0), ("dx", "dweight"))
        return
    run(parts(ints, 3, rows, width), sparse(signs(rows, d), 0), sparse(signs(2 * width, d), 0), ("dx", "dweight"))
    run(parts(ints, 2, rows, width), sparse(parts(ints, 2, rows, d), 0), sparse(parts(ints, 2, 2 * width, d), 0), ("dx", "dweight"))
    # few numbers of dpre along a row, for dx, and along a column, for dweight
    few = sparse(signs(rows, width), 1)
    few[:, torch.arange(width, device=DEV) % 2 == 1] = 0
    run(few, signs(rows, d), parts(ints, 3, 2 * width, d), ("dx",))
    run(sparse(signs(rows, width), 0), parts(ints, 3, rows, d), signs(2 * width, d), ("dweight",))


# ----------------------------------------------------- sizes of the numbers --

# float32's largest number, numbers past bfloat16's largest, all 24 bits set,
# down to parts of 2^-117
VALUES = [3.4028234663852886e38, -3.4e38, 3.39e38, 16777215.0, -3.1415927410125732, 1.0000001192092896, 2.0 ** -90 * (1 + 2.0 ** -23),
          -1e30, 1e-25]


def values(n):
    import torch
    v = torch.tensor(VALUES, device=DEV)
    return v[torch.arange(n, device=DEV) % len(VALUES)]


@pytest.mark.parametrize("rows,d,width", [(4100, 40, 33), (1301, 515, 1203), (300, 16384, 40), (3, 20, 9)])
def test_numbers_of_every_size(rows, d, width):
    """One number times a power of two in each sum: three parts that add up to
    it give it back, of any size; forward (split, and where few rows are read as
    they are), dx and dweight."""
    import torch
    k = torch.arange(rows, device=DEV) % d
    x = torch.zeros(rows, d, device=DEV)
    x[torch.arange(rows, device=DEV), k] = values(rows)
    w = 2.0 ** -(torch.arange(2 * width * d, device=DEV) % 5).float().view(2 * width, d)
    h, pre = nan((rows, width), torch.float32), nan((rows, 2 * width), torch.float32)
    la.kfac_gated_forward(x, w, h, pre=pre, activation="relu")
    assert torch.equal(pre, values(rows)[:, None] * w[:, k].t())
    # dpre = dh on the gates' side and on the other: one place of a row in W's columns, one row in x's
    dh = values(rows)[:, None].expand(rows, width).contiguous()
    w = torch.zeros(2 * width, d, device=DEV)
    j = torch.arange(d, device=DEV) % (2 * width)
    w[j, torch.arange(d, device=DEV)] = 2.0 ** -(torch.arange(d, device=DEV) % 5).float()
    x = torch.zeros(rows, d, device=DEV)
    i = torch.arange(d, device=DEV) % rows
    x[i, torch.arange(d, device=DEV)] = 2.0 ** -(torch.arange(d, device=DEV) % 3).float()
    dpre, dx, dw = nan((rows, 2 * width), torch.float32), nan((rows, d), torch.float32), nan((2 * width, d), torch.float32)
    la.kfac_gated_backward(dh, x, w, torch.ones(rows, 2 * width, device=DEV), dpre, dx, dw, activation="relu")
    assert torch.equal(dpre, torch.cat([dh, dh], 1))
    assert torch.equal(dx, values(rows)[:, None] * w.sum(0))
    assert torch.equal(dw, (values(rows)[i] * x[i, torch.arange(d, device=DEV)]).expand(2 * width, d))


def test_infinities_in_parts():
    """An infinity makes the sums that it enters infinite or NaN, and no others."""
    import torch
    rows, d, width = 4100, 40, 33
    assert la.load_library().kfac_gated_workspace_size(rows, d, width, la.KFAC_F32, 0) > 0
    _, ints = draw(9)
    x, w = ints(-1, 1, rows, d, dtype=torch.float32), ints(1, 2, 2 * width, d, dtype=torch.float32)
    h, pre, pre2 = nan((rows, width), torch.float32), nan((rows, 2 * width), torch.float32), nan((rows, 2 * width), torch.float32)
    la.kfac_gated_forward(x, w, h, pre=pre, activation="relu")
    x[4099, 39], x[7, 0] = float("inf"), float("-inf")
    la.kfac_gated_forward(x, w, h, pre=pre2, activation="relu")
    rest = [r for r in range(rows) if r not in (7, 4099)]
    assert torch.equal(pre2[rest], pre[rest]) and not bool(pre2[[7, 4099]].isfinite().any())
