"""Host side of layer norm and of gradient clipping: refusals of the C entry
points and of the binding (nothing reaches the GPU)."""
import ctypes
import struct

import pytest

import linear_algebra_amd as la

OK, INVALID, WORKSPACE = 0, 1, 2
FAKE = 1 << 20            # an aligned address that no refused call reads
REFUSED = ctypes.c_size_t(-1).value
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from linear_algebra_amd import build
    build.build()
    return la.load_library()


# ------------------------------------------------------------- layer norm --

def norm_forward(lib, rows=4, d=8, dtype=BF16, x=FAKE, sx=8, y=FAKE, sy=8, mean=FAKE, rstd=FAKE, w=FAKE, b=FAKE, kind=F32,
                 eps=1e-5):
    return lib.kfac_layer_norm_forward(rows, d, dtype, x, sx, y, sy, mean, rstd, w, b, kind, eps, None)


def norm_backward(lib, rows=4, d=8, dtype=BF16, dy=FAKE, sdy=8, x=FAKE, sx=8, mean=FAKE, rstd=FAKE, w=FAKE, dx=FAKE, sdx=8,
                  dw=FAKE, db=FAKE, kind=F32, ws=FAKE, size=1 << 30):
    return lib.kfac_layer_norm_backward(rows, d, dtype, dy, sdy, x, sx, mean, rstd, w, dx, sdx, dw, db, kind, ws, size, None)


BOTH = [dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=16385), dict(dtype=2), dict(kind=5), dict(dtype=F32, kind=BF16),
        dict(x=None), dict(x=FAKE + 1), dict(sx=7), dict(sx=-8), dict(mean=FAKE + 2), dict(rstd=FAKE + 1), dict(w=FAKE + 2),
        dict(dtype=F32, x=FAKE + 2)]


@pytest.mark.parametrize("bad", BOTH + [dict(y=None), dict(sy=3), dict(b=FAKE + 1), dict(eps=-1e-9), dict(eps=float("nan")),
                                        dict(eps=float("inf"))], ids=str)
def test_norm_forward_refuses(lib, bad):
    assert norm_forward(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", BOTH + [dict(dy=None), dict(sdy=0), dict(mean=None), dict(rstd=None), dict(dx=FAKE + 1),
                                        dict(sdx=7), dict(dw=FAKE + 2), dict(db=FAKE + 1)], ids=str)
def test_norm_backward_refuses(lib, bad):
    assert norm_backward(lib, **bad) == INVALID


def test_norm_workspace(lib):
    need = lib.kfac_layer_norm_workspace_size(4, 8)
    assert 0 < need < 1 << 20
    for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(size=need - 1)):
        assert norm_backward(lib, **bad) == WORKSPACE
    assert lib.kfac_layer_norm_workspace_size(-1, 8) == REFUSED == lib.kfac_layer_norm_workspace_size(4, 0)
    # what is not formed needs none, and without rows there is nothing to launch
    assert norm_backward(lib, rows=0, dw=None, db=None, ws=None, size=0) == OK
    assert norm_forward(lib, rows=0, x=None, y=None, mean=None, rstd=None) == OK


# --------------------------------------------------------- gradient norm --

def pointers(*at):
    return struct.pack(f"@{len(at)}P", *at)


def clip(lib, n=2, g=pointers(FAKE, FAKE + 64), out=pointers(FAKE, FAKE + 64), count=(4, 4), dtype=(F32, F32), max_norm=1.0,
         norm=FAKE + 4096, ws=FAKE, size=1 << 20):
    c = None if count is None else struct.pack(f"@{len(count)}q", *count)
    t = None if dtype is None else struct.pack(f"@{len(dtype)}i", *dtype)
    return lib.kfac_grad_clip(n, g, out, c, t, max_norm, norm, ws, size, None)


@pytest.mark.parametrize("bad", [dict(n=0), dict(n=4097), dict(g=None), dict(out=None), dict(count=None), dict(dtype=None),
                                 dict(count=(4, -1)), dict(count=(4, 1 << 38)), dict(dtype=(F32, 3)), dict(norm=None),
                                 dict(norm=FAKE + 2), dict(max_norm=-1.0), dict(max_norm=float("nan")),
                                 dict(g=pointers(FAKE, 0)), dict(out=pointers(FAKE, 0)), dict(g=pointers(FAKE + 2, FAKE + 64)),
                                 dict(dtype=(F32, BF16), out=pointers(FAKE, FAKE + 65))], ids=str)
def test_clip_refuses(lib, bad):
    assert clip(lib, **bad) == INVALID
    if not {"out", "max_norm"} & set(bad):
        n = bad.get("n", 2)
        c, t = bad.get("count", (4, 4)), bad.get("dtype", (F32, F32))
        assert lib.kfac_grad_norm(n, bad.get("g", pointers(FAKE, FAKE + 64)), c and struct.pack("@2q", *c),
                                  t and struct.pack("@2i", *t), bad.get("norm", FAKE), FAKE, 1 << 20, None) == INVALID


@pytest.mark.parametrize("g,out", [((0, 0), (0, 0)), ((0, 12), (0, 12)), ((12, 0), (12, 0)), ((0, 64), (64, 0)),
                                   ((0, 64), (4, 64)), ((0, 64), (0, 60)), ((0, 64), (128, 140)), ((64, 0), (64, 52))])
def test_clip_refuses_overlaps(lib, g, out):
    assert clip(lib, g=pointers(*(FAKE + k for k in g)), out=pointers(*(FAKE + k for k in out))) == INVALID


@pytest.mark.parametrize("at", [0, 12, 64, 76, 128, 140, 192, 204])
def test_clip_refuses_a_norm_inside_a_tensor(lib, at):
    where = dict(g=pointers(FAKE, FAKE + 64), out=pointers(FAKE + 128, FAKE + 192))
    assert clip(lib, norm=FAKE + at, **where) == INVALID
    assert clip(lib, norm=FAKE + 16, size=64, **where) == WORKSPACE


def test_clip_workspace(lib):
    need = lib.kfac_grad_norm_workspace_size(4096)
    assert 0 < need < 1 << 20
    assert lib.kfac_grad_norm_workspace_size(0) == REFUSED == lib.kfac_grad_norm_workspace_size(4097)
    for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(size=64)):
        assert clip(lib, **bad) == WORKSPACE


# ----------------------------------------------------------------- binding --

def test_binding_refuses_host_tensors():
    import torch
    x, v, m = torch.zeros(4, 8), torch.ones(8), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        la.kfac_layer_norm_forward(x, x.clone(), m, m.clone(), weight=v)
    with pytest.raises(ValueError, match="GPU"):
        la.kfac_layer_norm_backward(x, x, m, m, x.clone())
    with pytest.raises(ValueError, match="GPU"):
        la.kfac_grad_clip([x], 1.0, torch.zeros(1))
    with pytest.raises(ValueError, match="at least one"):
        la.kfac_grad_norm([], torch.zeros(1))
    with pytest.raises(TypeError):
        la.kfac_grad_norm([x, None], torch.zeros(1))
    with pytest.raises(TypeError):
        la.kfac_layer_norm_forward(None, x)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        la.kfac_layer_norm_forward(x.double(), x.double())


def test_shapes_are_checked_before_the_kernels():
    import torch
    from linear_algebra_amd import training
    with pytest.raises(ValueError, match="shape"):
        training.layer_norm(torch.zeros(3, 8), torch.ones(7))
    with pytest.raises(ValueError, match="shape"):
        training.layer_norm(torch.zeros(8), torch.ones(8, 8), dims=2)
    with pytest.raises(ValueError, match="last dimensions"):
        training.LayerNorm(6)(torch.zeros(3, 8))


def test_no_gradients_have_no_norm():
    import torch
    from linear_algebra_amd import training
    assert float(training.clip_grad_norm_([torch.nn.Parameter(torch.ones(3))], 1.0)) == 0.0
    assert float(training.clip_grad_norm_([], 1.0)) == 0.0


# ------------------------------------------------------------------- gated --

def gated_forward(lib, rows=4, d=8, width=6, dtype=BF16, act=0, x=FAKE, w=FAKE, b=FAKE, h=FAKE, pre=FAKE, ws=FAKE, size=1 << 40):
    return lib.kfac_gated_forward(rows, d, width, dtype, act, x, w, b, h, pre, ws, size, None)


def gated_backward(lib, rows=4, d=8, width=6, dtype=BF16, act=0, dh=FAKE, x=FAKE, w=FAKE, pre=FAKE, dpre=FAKE, dx=FAKE, dw=FAKE,
                   kind=F32, db=FAKE, ws=FAKE, size=1 << 40):
    return lib.kfac_gated_backward(rows, d, width, dtype, act, dh, x, w, pre, dpre, dx, dw, kind, db, ws, size, None)


GATED = [dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=16385), dict(width=0), dict(width=16385), dict(dtype=2), dict(act=-1),
         dict(act=5), dict(x=None), dict(x=FAKE + 2), dict(w=None), dict(w=FAKE + 2), dict(pre=FAKE + 1), dict(dtype=F32, x=FAKE + 2)]


@pytest.mark.parametrize("bad", GATED + [dict(h=None), dict(h=FAKE + 1), dict(b=FAKE + 2), dict(dtype=F32, h=FAKE + 2)], ids=str)
def test_gated_forward_refuses(lib, bad):
    assert gated_forward(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", GATED + [dict(dh=None), dict(dh=FAKE + 1), dict(pre=None), dict(dpre=None), dict(dpre=FAKE + 2),
                                         dict(dx=FAKE + 1), dict(dw=FAKE + 2), dict(kind=3), dict(dtype=F32, kind=BF16),
                                         dict(db=FAKE + 2)], ids=str)
def test_gated_backward_refuses(lib, bad):
    assert gated_backward(lib, **bad) == INVALID


def test_gated_workspace(lib):
    for bad in ((-1, 8, 6, BF16), (4, 0, 6, BF16), (4, 8, 16385, BF16), (4, 8, 6, 7)):
        for way in (0, 1):
            assert lib.kfac_gated_workspace_size(*bad, way) == REFUSED
    # bfloat16 of even width is read as it is, and so are few rows; what else goes through copies
    for sizes in ((4000, 64, 600, BF16), (4, 9, 6, BF16), (4, 8, 6, F32)):
        assert lib.kfac_gated_workspace_size(*sizes, 0) == 0
    for sizes in ((4000, 9, 600, BF16), (4000, 8, 600, F32)):
        need = lib.kfac_gated_workspace_size(*sizes, 0)
        assert need > 0
        for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(size=need - 1)):
            assert gated_forward(lib, *sizes, **bad) == WORKSPACE
    need = lib.kfac_gated_workspace_size(4, 8, 6, BF16, 1)
    assert need > 0 and gated_backward(lib, size=need - 1) == WORKSPACE


def test_gated_binding_refuses():
    import torch
    x, w, h, p = torch.zeros(4, 8), torch.zeros(12, 8), torch.zeros(4, 6), torch.zeros(4, 12)
    with pytest.raises(ValueError, match="GPU"):
        la.kfac_gated_forward(x, w, h)
    with pytest.raises(ValueError, match="GPU"):
        la.kfac_gated_backward(h, x, w, p, p.clone())
    with pytest.raises(TypeError):
        la.kfac_gated_forward(x, None, h)
