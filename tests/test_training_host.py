"""Host side of the encoder-layer training operators: refusals of the C entry
points and of the binding (nothing reaches the GPU), the bucket borders, and
the float64 forms the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import linear_algebra_amd as la
from tests import training_reference as ref

OK, INVALID, WORKSPACE = 0, 1, 2
FAKE = 1 << 20            # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    from linear_algebra_amd import build
    build.build()
    return la.load_library()


class Attention(ctypes.Structure):
    """kfac_attention_t"""
    _fields_ = [("batch", ctypes.c_int64), ("len_q", ctypes.c_int64), ("len_k", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
                ("n_borders", ctypes.c_int32), ("two_sided", ctypes.c_int32),
                ("borders", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class Tensor4(ctypes.Structure):
    """kfac_tensor4_t"""
    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_int64), ("stride_row", ctypes.c_int64),
                ("stride_head", ctypes.c_int64)]


REFUSED = ctypes.c_size_t(-1).value


def test_packed_forms_match_the_structs():
    assert la._ATTENTION.size == ctypes.sizeof(Attention) and la._TENSOR4.size == ctypes.sizeof(Tensor4)
    raw = la._ATTENTION.pack(1, 2, 3, 4, 5, 6, 7, 0.5, 8, 9, 10, 11, 12)
    f = Attention.from_buffer_copy(raw)
    assert [getattr(f, n) for n, _ in f._fields_] == [1, 2, 3, 4, 5, 6, 7, 0.5, 8, 9, 10, 11, 12]


def form(**kw):
    f = Attention(2, 8, 8, 4, 2, 16, 0, 0.25, 0, 1, None, None, None)
    for k, v in kw.items():
        setattr(f, k, v)
    return f


def tensor(heads=4, **kw):
    t = Tensor4(FAKE, 8 * heads * 16, heads * 16, 16)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def fwd(lib, f, ws=FAKE, ws_bytes=1 << 30, dtype=1, q=None, k=None, lse=FAKE):
    q, k, v, o = q or tensor(), k or tensor(2), tensor(2), tensor()
    return lib.kfac_attention_forward(ctypes.byref(f), dtype, ctypes.byref(q), ctypes.byref(k), ctypes.byref(v),
                                      ctypes.byref(o), lse, ws, ws_bytes, None)


BAD_FORMS = [dict(batch=-1), dict(len_q=-1), dict(len_k=(1 << 24) + 1), dict(heads=0), dict(heads=3), dict(kv_heads=0),
             dict(dim=4), dict(dim=12), dict(dim=136), dict(scale=0.0), dict(scale=float("nan")),
             dict(scale=float("inf")), dict(scale=-1.0), dict(lens=FAKE + 1), dict(batch=1 << 40),
             dict(bias=FAKE, n_borders=-1), dict(bias=FAKE, n_borders=3), dict(bias=FAKE, n_borders=64)]


@pytest.mark.parametrize("bad", BAD_FORMS, ids=str)
def test_attention_refuses_forms(lib, bad):
    f = form(**bad)
    if bad.get("n_borders", 0) == 64:
        at = (ctypes.c_int32 * 64)(*range(1, 65))
        f.borders = ctypes.addressof(at)
    for backward in (0, 1):
        assert lib.kfac_attention_workspace_size(ctypes.byref(f), 1, backward) == REFUSED
    assert fwd(lib, f) == INVALID


@pytest.mark.parametrize("borders", [[0], [2, 2], [3, 1], [-1], [1 << 30]])
def test_attention_refuses_borders(lib, borders):
    at = (ctypes.c_int32 * len(borders))(*borders)
    f = form(bias=FAKE, n_borders=len(borders), borders=ctypes.addressof(at))
    assert lib.kfac_attention_workspace_size(ctypes.byref(f), 1, 0) == REFUSED
    assert fwd(lib, f) == INVALID


def test_attention_refuses_tensors(lib):
    f = form()
    assert fwd(lib, f, dtype=7) == INVALID
    assert fwd(lib, f, lse=None) == INVALID
    # a stretch of distances too long for LDS needs a workspace
    at = (ctypes.c_int32 * 2)(1, 5000)
    wide = form(bias=FAKE, n_borders=2, borders=ctypes.addressof(at))
    assert lib.kfac_attention_workspace_size(ctypes.byref(wide), 1, 0) > 0
    assert lib.kfac_attention_workspace_size(ctypes.byref(f), 1, 0) == 0
    assert lib.kfac_attention_workspace_size(ctypes.byref(f), 5, 0) == REFUSED
    for bad in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=0)):
        assert fwd(lib, wide, **bad) == WORKSPACE
    for bad in (dict(data=None), dict(data=FAKE + 8), dict(stride_row=60), dict(stride_row=-64), dict(stride_batch=4),
                dict(stride_head=-16), dict(stride_row=1 << 23)):
        assert fwd(lib, f, q=tensor(**bad)) == INVALID, bad
        assert fwd(lib, f, k=tensor(2, **bad)) == INVALID, bad
    assert lib.kfac_attention_forward(None, 1, None, None, None, None, None, None, 0, None) == INVALID


def test_attention_backward_refuses(lib):
    at = (ctypes.c_int32 * 1)(3)
    biased = form(bias=FAKE, n_borders=1, borders=ctypes.addressof(at))
    for f, dbias in ((form(), FAKE), (biased, None), (biased, FAKE + 2)):
        ts = [tensor(4 if n in (0, 3, 4, 5) else 2) for n in range(8)]
        r = [ctypes.byref(t) for t in ts]
        assert lib.kfac_attention_backward(ctypes.byref(f), 1, r[0], r[1], r[2], r[3], FAKE, r[4], r[5], r[6], r[7], dbias,
                                           FAKE, 1 << 30, None) == INVALID
    ts = [ctypes.byref(tensor(4 if n in (0, 3, 4, 5) else 2)) for n in range(8)]
    assert lib.kfac_attention_workspace_size(ctypes.byref(biased), 1, 1) > 0
    for ws, size in ((None, 1 << 30), (FAKE + 8, 1 << 30), (FAKE, 8)):
        assert lib.kfac_attention_backward(ctypes.byref(biased), 1, ts[0], ts[1], ts[2], ts[3], FAKE, ts[4], ts[5], ts[6],
                                           ts[7], FAKE, ws, size, None) == WORKSPACE


def test_attention_with_nothing_to_do_needs_no_gpu(lib):
    for f in (form(batch=0), form(len_q=0)):
        assert fwd(lib, f) == OK


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def ptr(*v):
    return (ctypes.c_void_p * len(v))(*v)


def test_checkpoint_refusals(lib):
    good = dict(n=1, x=ptr(FAKE), rows=i64(5), d=i64(7), ones=1, dtype=0, codes=ptr(FAKE), scales=ptr(FAKE))
    bad = [dict(n=0), dict(n=4097), dict(x=None), dict(x=ptr(None)), dict(x=ptr(FAKE + 2)), dict(rows=i64(0)),
           dict(rows=i64(1 << 31)), dict(d=i64(0)), dict(d=i64(16384)), dict(ones=2), dict(dtype=5), dict(codes=ptr(None)),
           dict(codes=ptr(FAKE + 8)), dict(scales=ptr(None))]
    for b in bad:
        a = dict(good, **b)
        assert lib.kfac_checkpoint_store(a["n"], a["x"], a["rows"], a["d"], a["ones"], a["dtype"], a["codes"], a["scales"],
                                         None) == INVALID, b
    load = dict(n=1, codes=ptr(FAKE), scales=ptr(FAKE), rows=i64(5), d=i64(7), cols=i64(7), dtype=1, y=ptr(FAKE))
    for b in (dict(cols=i64(0)), dict(cols=i64(8)), dict(y=ptr(None)), dict(y=ptr(FAKE + 1)), dict(codes=ptr(FAKE + 4)),
              dict(rows=i64(0)), dict(dtype=-1), dict(d=None)):
        a = dict(load, **b)
        assert lib.kfac_checkpoint_load(a["n"], a["codes"], a["scales"], a["rows"], a["d"], a["cols"], a["dtype"], a["y"],
                                        None) == INVALID, b
    fac = dict(n=1, codes=ptr(FAKE), scales=ptr(FAKE), rows=i64(4096), d=i64(7), m=ptr(FAKE), eps=0.5, ws=FAKE, b=1 << 30)
    for b, want in ((dict(eps=1.5), INVALID), (dict(eps=float("nan")), INVALID), (dict(m=ptr(FAKE + 2)), INVALID),
                    (dict(rows=i64(0)), INVALID), (dict(d=i64(16385)), INVALID), (dict(ws=None), WORKSPACE),
                    (dict(ws=FAKE + 16), WORKSPACE), (dict(b=8), WORKSPACE)):
        a = dict(fac, **b)
        assert lib.kfac_checkpoint_factors(a["n"], a["codes"], a["scales"], a["rows"], a["d"], a["m"], a["eps"], 1, a["ws"],
                                           a["b"], None) == want, b
    grad = dict(n=1, g=ptr(FAKE), codes=ptr(FAKE), scales=ptr(FAKE), rows=i64(4096), o=i64(3), d=i64(7), dtype=0,
                mat=ptr(FAKE), ws=FAKE, b=1 << 30)
    for b, want in ((dict(o=i64(0)), INVALID), (dict(o=i64(16385)), INVALID), (dict(g=ptr(FAKE + 2)), INVALID),
                    (dict(mat=ptr(None)), INVALID), (dict(dtype=9), INVALID), (dict(b=0), WORKSPACE)):
        a = dict(grad, **b)
        assert lib.kfac_checkpoint_grad(a["n"], a["g"], a["codes"], a["scales"], a["rows"], a["o"], a["d"], a["dtype"],
                                        a["mat"], a["ws"], a["b"], None) == want, b
    assert lib.kfac_checkpoint_factors_workspace_size(0, i64(1), i64(1)) == REFUSED
    assert lib.kfac_checkpoint_grad_workspace_size(1, i64(1), i64(0), i64(1)) == REFUSED
    assert lib.kfac_checkpoint_factors_workspace_size(1, i64(5), i64(7)) == 0


def test_binding_refuses_host_tensors_and_shapes(lib):
    import torch
    q = torch.zeros(1, 4, 2, 16)
    with pytest.raises(ValueError, match="on the GPU"):
        la.kfac_attention_forward(q, q, q, q, torch.zeros(1, 2, 4))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        la.kfac_attention_forward(q.half(), q, q, q, torch.zeros(1, 2, 4))
    with pytest.raises(TypeError):
        la.kfac_attention_forward(None, q, q, q, q)
    c, s = la.kfac_checkpoint_empty(33, 5, "cpu")
    assert c.shape == (2, 5, 32) and s.shape == (2, 5)
    with pytest.raises(ValueError, match="on the GPU"):
        la.kfac_checkpoint_store([torch.zeros(33, 5)], [c], [s])
    with pytest.raises(ValueError, match="equally many"):
        la.kfac_checkpoint_store([torch.zeros(33, 5)], [], [])
    with pytest.raises(ValueError):
        la.kfac_checkpoint_store([], [], [])
    with pytest.raises(ValueError, match="two-dimensional"):
        la.kfac_checkpoint_grad([torch.zeros(33)], [c], [s], [c])


def test_position_borders():
    assert la.kfac_position_borders(1, 100) == []
    assert la.kfac_position_borders(8, 128) == [1, 2, 3, 4, 10, 23, 54]
    for n, far in ((16, 128), (32, 1024), (31, 500), (64, 40)):
        b = la.kfac_position_borders(n, far)
        assert len(b) == n - 1 and all(x < y for x, y in zip(b, b[1:])) and b[0] == 1
        near, wide = n // 2, n - n // 2
        for m in range(1, wide):
            t = b[near + m - 1]
            if t > b[near + m - 2] + 1:    # the least distance that qualifies
                assert t ** wide * near ** m >= far ** m * near ** wide > (t - 1) ** wide * near ** m
    for n, far in ((0, 5), (8, 4)):
        with pytest.raises(ValueError):
            la.kfac_position_borders(n, far)


def test_reference_gradients_against_differences():
    """The float64 gradient formulas the GPU tests use, against central
    differences of the float64 forward: h^2 / 6 of the third derivative
    (order one) at h = 1e-4, and float64 rounding over h."""
    import torch
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 5, 4, 8, generator=g, dtype=torch.float64)
    k, v = (torch.randn(2, 7, 2, 8, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(2, 5, 4, 8, generator=g, dtype=torch.float64)
    borders = [1, 2, 4]
    kw = dict(scale=8 ** -0.5, causal=True, lens=torch.tensor([7, 4]), borders=borders, two_sided=True)
    x = {"q": q, "k": k, "v": v, "bias": torch.randn(8, 4, generator=g, dtype=torch.float64)}

    def run(x):
        return ref.attention(x["q"], x["k"], x["v"], bias=x["bias"], **kw)

    f = run(x)
    got = ref.attention(x["q"], x["k"], x["v"], bias=x["bias"], out=f["out"][0], lse=f["lse"][0], dout=w, **kw)
    h = 1e-4
    for n in x:
        d = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
        r = [float((run(dict(x, **{n: x[n] + s * h * d}))["out"][0] * w).sum()) for s in (1, -1)]
        formula = float((got["d" + n][0] * d).sum())
        assert abs((r[0] - r[1]) / (2 * h) - formula) <= 1e-6 * max(1.0, abs(formula))


def test_reference_codes():
    """The 8-bit form against its definition: every code's value is its own nearest, ties go to the even code."""
    codes = np.arange(256, dtype=np.uint8)
    fin = codes[(codes & 0x7f) != 0x7f]
    v = ref.decode(np.broadcast_to(fin[None, :, None], (1, fin.size, 32)).copy(), np.full((1, fin.size), 127, np.uint8), 32)[0]
    assert v.max() == 448.0 and v.min() == -448.0
    full = np.zeros((32, fin.size))
    full[0], full[1] = v, 448.0
    c, s = ref.encode(full, False)
    assert np.all(s == 127) and np.array_equal(c[0, :, 0], fin)
    pos = np.sort(v[v >= 0])[1:]
    mid = (pos[1:] + pos[:-1]) / 2
    full = np.zeros((32, mid.size))
    full[0], full[1] = mid, 448.0
    c, _ = ref.encode(full, False)
    assert np.all(c[0, :, 0] % 2 == 0)
    c, s = ref.encode(np.full((1, 1), 449.0), True)
    assert s.tolist() == [[128, 119]] and c[0, 1, 0] == 0x78 and not c[0, :, 1:].any()


def path_of(lib, case):
    """Which kernels a case of tests/test_gpu_attention.py takes, from the
    workspace it is given: queries per workgroup of the passes by queries,
    shares of the key tiles, and whether the bias is looked up in memory."""
    dtype, b, lq, lk, h, hk, d, causal, two_sided, borders, lens = case
    at = (ctypes.c_int32 * max(1, len(borders or [])))(*(borders or []))

    def size(backward, bias, n, two):
        f = form(batch=b, len_q=lq, len_k=lk, heads=h, kv_heads=hk, dim=d, causal=int(causal), two_sided=two,
                 bias=FAKE if bias else None, n_borders=n, borders=ctypes.addressof(at) if n else None)
        got = lib.kfac_attention_workspace_size(ctypes.byref(f), 1 if dtype == "bf16" else 0, backward)
        assert got != REFUSED
        return got

    def room(*floats):
        return sum((4 * n + 255) // 256 * 256 for n in floats)

    plain = size(1, False, 0, 0)
    stats = 2 * b * h * ((lq + 127) // 128 * 128)
    shares = (plain - room(stats)) // (4 * 2 * b * hk * lk * d)
    per = size(1, True, 0, 0) - plain          # one bucket: a float per wave of the pass by queries
    rows = [n for n in (32, 128) if room(b * h * ((lq + n - 1) // n) * 4) == per]
    memory = borders is not None and size(0, True, len(borders), int(two_sided)) > 0
    return rows, max(1, shares), memory


def test_paths_of_the_gpu_tests(lib):
    """The cases that are there to test a path still take it."""
    from tests import test_gpu_attention as t
    for case in t.WIDE:
        assert path_of(lib, case)[0] == [128], case
    for case in t.UNSHARED:
        rows, shares, _ = path_of(lib, case)
        assert 128 in rows and shares == 1, case
    for dtype in ("bf16", "f32"):
        # 128 queries per workgroup at every head width that has kernels of its own, with and without a bias
        # from memory; unshared key tiles likewise
        wide = [c for c in t.WIDE if c[0] == dtype]
        assert {(c[6] + 31) // 32 for c in wide} == {1, 2, 3, 4}
        assert {path_of(lib, c)[2] for c in wide} == {False, True}
        assert {c[9] is None for c in wide} == {False, True} and {c[7] for c in wide} == {False, True}
        one = [c for c in t.UNSHARED if c[0] == dtype]
        assert len({(c[6] + 31) // 32 for c in one}) >= 3 and {path_of(lib, c)[2] for c in one} == {False, True}
    # 32 queries per workgroup, and shared key tiles, among the older cases
    assert all(32 in path_of(lib, c)[0] for c in t.CASES)
    assert sum(path_of(lib, c)[1] > 1 for c in t.CASES) >= 10
