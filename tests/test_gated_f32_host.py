"""Host side of the gated backward pass of bfloat16 rows with a float32 dpre:
refusals and workspace (nothing reaches the GPU)."""
import ctypes

import pytest

import linear_algebra_amd as la

INVALID, WORKSPACE = 1, 2
FAKE = 1 << 20            # an aligned address that no refused call reads
REFUSED = ctypes.c_size_t(-1).value
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from linear_algebra_amd import build
    build.build()
    return la.load_library()


def backward(lib, rows=4, d=8, width=6, act=0, dh=FAKE, x=FAKE, w=FAKE, pre=FAKE, dpre=FAKE, dx=FAKE, dw=FAKE, kind=F32, db=FAKE,
             ws=FAKE, size=1 << 40):
    return lib.kfac_gated_backward_f32(rows, d, width, act, dh, x, w, pre, dpre, dx, dw, kind, db, ws, size, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=1 << 31), dict(d=0), dict(d=16385), dict(width=0), dict(width=16385),
                                 dict(act=-1), dict(act=5), dict(dh=None), dict(dh=FAKE + 1), dict(x=None), dict(x=FAKE + 2),
                                 dict(w=None), dict(w=FAKE + 2), dict(pre=None), dict(pre=FAKE + 1), dict(dpre=None),
                                 dict(dpre=FAKE + 2), dict(dx=FAKE + 1), dict(dw=FAKE + 2), dict(kind=3), dict(db=FAKE + 2)],
                         ids=str)
def test_refuses(lib, bad):
    assert backward(lib, **bad) == INVALID


def test_workspace(lib):
    assert lib.kfac_gated_workspace_size(4, 8, 16385, BF16, 2) == REFUSED
    for sizes in ((4, 8, 6), (4000, 64, 600), (3, 9, 5)):
        need = lib.kfac_gated_workspace_size(*sizes, BF16, 2)
        # dpre's three parts at least
        assert need >= 3 * 2 * sizes[0] * 2 * sizes[2]
        for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(size=64)):
            assert backward(lib, *sizes, **bad) == WORKSPACE


def test_binding_refuses():
    import torch
    x, w, h, p = (torch.zeros(s).bfloat16() for s in ((4, 8), (12, 8), (4, 6), (4, 12)))
    with pytest.raises(ValueError, match="GPU"):
        la.kfac_gated_backward(h, x, w, p, p.float())
