"""Python binding of the MI355X K-FAC hot-path library (libkfac.so).

The functions here carry the names of the C entry points in include/kfac.h
and do argument marshalling only: they check tensor shapes, dtypes and
devices, gather data pointers, take a workspace from PyTorch's allocator and
pass the current HIP stream.  Every step of the computation runs in the HIP
kernels of libkfac.so; there is no fallback.  If the library is missing the
import of this package succeeds but every call raises ``KfacLibraryError``.

PyTorch provides device memory and streams only.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkfac.so")

KFAC_OK, KFAC_ERR_INVALID_VALUE, KFAC_ERR_WORKSPACE, KFAC_ERR_UNSUPPORTED, KFAC_ERR_HIP = range(5)
KFAC_F32, KFAC_BF16 = 0, 1
KFAC_PACK, KFAC_UNPACK = 0, 1

EXPORTS = (
    "kfac_abi_version", "kfac_status_string",
    "kfac_factors_workspace_size", "kfac_factors",
    "kfac_packed_size", "kfac_pack_workspace_size", "kfac_pack_sym", "kfac_pack_sym_static", "kfac_stream_copy",
    "kfac_matrix_rate",
    "kfac_inverse_workspace_size", "kfac_damped_inverse",
    "kfac_precondition_workspace_size", "kfac_precondition",
    "kfac_im2col_workspace_size", "kfac_im2col",
    "kfac_grad_rows_workspace_size", "kfac_grad_rows",
    "kfac_grad_matrix_workspace_size", "kfac_grad_matrix",
    "kfac_attention_workspace_size", "kfac_attention_forward", "kfac_attention_backward",
    "kfac_checkpoint_store", "kfac_checkpoint_load",
    "kfac_checkpoint_factors_workspace_size", "kfac_checkpoint_factors",
    "kfac_checkpoint_grad_workspace_size", "kfac_checkpoint_grad",
    "kfac_layer_norm_forward", "kfac_layer_norm_workspace_size", "kfac_layer_norm_backward",
    "kfac_gated_workspace_size", "kfac_gated_forward", "kfac_gated_backward", "kfac_gated_backward_f32",
    "kfac_grad_norm_workspace_size", "kfac_grad_norm", "kfac_grad_clip",
)


class KfacConv(ctypes.Structure):
    """kfac_conv_t: shape of a layer input and its convolution (1 x 1 for a
    fully connected layer)."""
    _fields_ = [("n", ctypes.c_int64), ("c", ctypes.c_int64), ("h", ctypes.c_int64), ("w", ctypes.c_int64),
                ("kh", ctypes.c_int32), ("kw", ctypes.c_int32), ("sh", ctypes.c_int32), ("sw", ctypes.c_int32),
                ("ph", ctypes.c_int32), ("pw", ctypes.c_int32), ("dh", ctypes.c_int32), ("dw", ctypes.c_int32),
                ("ones", ctypes.c_int32), ("reserved", ctypes.c_int32)]


# kfac_attention_t and kfac_tensor4_t as packed bytes (the library reads them during the call only)
_ATTENTION = struct.Struct("@qqqiiiifiiPPP")
_TENSOR4 = struct.Struct("@Pqqq")


class KfacLibraryError(RuntimeError):
    pass


class KfacError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where} failed: {status_string(status)} ({status})")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libkfac.so and declare its C signatures (no GPU needed)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise KfacLibraryError(f"{path} is missing: build it with `python -m linear_algebra_amd.build`")
    lib = ctypes.CDLL(path)
    i32, i64, sz, vp, f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    sig = {
        "kfac_abi_version": (i32, []),
        "kfac_status_string": (ctypes.c_char_p, [i32]),
        "kfac_factors_workspace_size": (sz, [i32, vp, vp, i32]),
        "kfac_factors": (i32, [i32, vp, vp, vp, i32, vp, f32, i32, vp, sz, vp]),
        "kfac_packed_size": (i64, [i32, vp]),
        "kfac_pack_workspace_size": (sz, [i32, vp]),
        "kfac_pack_sym": (i32, [i32, vp, vp, vp, i32, vp, sz, vp]),
        "kfac_pack_sym_static": (i32, [i32, vp, vp, vp, i32, vp]),
        "kfac_stream_copy": (i32, [vp, vp, sz, vp]),
        "kfac_matrix_rate": (i32, [i32, i64, i32, vp, vp, vp]),
        "kfac_inverse_workspace_size": (sz, [i32, vp]),
        "kfac_damped_inverse": (i32, [i32, vp, vp, f32, vp, vp, vp, sz, vp]),
        "kfac_precondition_workspace_size": (sz, [i32, vp, vp]),
        "kfac_precondition": (i32, [i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "kfac_im2col_workspace_size": (sz, [i32]),
        "kfac_im2col": (i32, [i32, vp, vp, i32, vp, vp, sz, vp]),
        "kfac_grad_rows_workspace_size": (sz, [i32]),
        "kfac_grad_rows": (i32, [i32, vp, vp, vp, vp, i32, f32, vp, vp, sz, vp]),
        "kfac_grad_matrix_workspace_size": (sz, [i32]),
        "kfac_grad_matrix": (i32, [i32, vp, vp, vp, vp, vp, i32, vp, sz, vp]),
        "kfac_attention_workspace_size": (sz, [vp, i32, i32]),
        "kfac_attention_forward": (i32, [vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "kfac_attention_backward": (i32, [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "kfac_checkpoint_store": (i32, [i32, vp, vp, vp, i32, i32, vp, vp, vp]),
        "kfac_checkpoint_load": (i32, [i32, vp, vp, vp, vp, vp, i32, vp, vp]),
        "kfac_checkpoint_factors_workspace_size": (sz, [i32, vp, vp]),
        "kfac_checkpoint_factors": (i32, [i32, vp, vp, vp, vp, vp, f32, i32, vp, sz, vp]),
        "kfac_checkpoint_grad_workspace_size": (sz, [i32, vp, vp, vp]),
        "kfac_checkpoint_grad": (i32, [i32, vp, vp, vp, vp, vp, vp, i32, vp, vp, sz, vp]),
        "kfac_layer_norm_forward": (i32, [i64, i64, i32, vp, i64, vp, i64, vp, vp, vp, vp, i32, f32, vp]),
        "kfac_layer_norm_workspace_size": (sz, [i64, i64]),
        "kfac_layer_norm_backward": (i32, [i64, i64, i32, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, i32, vp, sz, vp]),
        "kfac_gated_workspace_size": (sz, [i64, i64, i64, i32, i32]),
        "kfac_gated_forward": (i32, [i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "kfac_gated_backward": (i32, [i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, sz, vp]),
        "kfac_gated_backward_f32": (i32, [i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, sz, vp]),
        "kfac_grad_norm_workspace_size": (sz, [i32]),
        "kfac_grad_norm": (i32, [i32, vp, vp, vp, vp, vp, sz, vp]),
        "kfac_grad_clip": (i32, [i32, vp, vp, vp, vp, f32, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().kfac_status_string(int(status)).decode()
    except KfacLibraryError:
        return str(status)


# ------------------------------------------------------------ marshalling --

def _i64(values) -> ctypes.Array:
    values = [int(v) for v in values]
    return (ctypes.c_int64 * len(values))(*values)


def _ptrs(tensors) -> ctypes.Array:
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _stream(device, stream):
    import torch
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the current stream's handle without building a Stream object (a tenth of the time)
    index = device.index
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index))


def _on(stream):
    """Workspaces come from torch's allocator on the stream that the call runs
    on: a block of another stream may still be in use by that one's earlier
    work, and may be handed out again there while this call's kernels use it."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _check(tensors, dtype, name):
    import torch
    dev = None
    for t in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected torch tensors")
        if t.device.type != "cuda":
            raise ValueError(f"{name}: tensors must live on the GPU")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name}: all tensors must be on one device")
    return dev


def _workspace(nbytes: int, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _call(status: int, where: str):
    if status != KFAC_OK:
        raise KfacError(status, where)


# ------------------------------------------------------------ entry points --

def kfac_factors(xs: Sequence, ms: Sequence, eps: float, first_step: bool, stream=None) -> None:
    """M_i <- F_i (first step) or eps*M_i + (1-eps)*F_i, F_i = x_i^T x_i / rows_i,
    upper triangle of each float32 M_i; x_i float32 or bfloat16 [rows_i, d_i]."""
    import torch
    lib = load_library()
    if len(xs) != len(ms) or len(xs) == 0:
        raise ValueError("kfac_factors: need equally many inputs and factors")
    dt = xs[0].dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("kfac_factors: inputs must be float32 or bfloat16")
    dev = _check(list(xs), dt, "kfac_factors(x)")
    _check(list(ms), torch.float32, "kfac_factors(m)")
    rows, d = [], []
    for x, m in zip(xs, ms):
        if x.dim() != 2 or m.shape != (x.shape[1], x.shape[1]):
            raise ValueError("kfac_factors: x must be [rows, d] and m [d, d]")
        rows.append(x.shape[0])
        d.append(x.shape[1])
    n = len(xs)
    r64, d64 = _i64(rows), _i64(d)
    dtype = KFAC_BF16 if dt == torch.bfloat16 else KFAC_F32
    ws_bytes = lib.kfac_factors_workspace_size(n, r64, d64, dtype)
    if ws_bytes == 0:
        raise KfacError(KFAC_ERR_INVALID_VALUE, "kfac_factors_workspace_size")
    with _on(stream):
        ws = _workspace(ws_bytes, dev)
    _call(lib.kfac_factors(n, _ptrs(xs), r64, d64, dtype, _ptrs(ms), ctypes.c_float(eps), int(bool(first_step)),
                           ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(dev, stream)), "kfac_factors")


def kfac_packed_size(dims: Sequence[int]) -> int:
    lib = load_library()
    v = lib.kfac_packed_size(len(dims), _i64(dims))
    if v < 0:
        raise KfacError(KFAC_ERR_INVALID_VALUE, "kfac_packed_size")
    return int(v)


def kfac_pack_sym(ms: Sequence, packed, direction: int, stream=None) -> None:
    """KFAC_PACK: upper triangles of ms -> packed.  KFAC_UNPACK: packed -> ms (both triangles)."""
    import torch
    lib = load_library()
    dev = _check(list(ms) + [packed], torch.float32, "kfac_pack_sym")
    d = []
    for m in ms:
        if m.dim() != 2 or m.shape[0] != m.shape[1]:
            raise ValueError("kfac_pack_sym: factors must be square")
        d.append(m.shape[0])
    n = len(ms)
    d64 = _i64(d)
    if packed.numel() != kfac_packed_size(d):
        raise ValueError("kfac_pack_sym: packed buffer has the wrong length")
    ws_bytes = lib.kfac_pack_workspace_size(n, d64)
    with _on(stream):
        ws = _workspace(ws_bytes, dev)
    _call(lib.kfac_pack_sym(n, _ptrs(ms), d64, ctypes.c_void_p(packed.data_ptr()), int(direction),
                            ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(dev, stream)), "kfac_pack_sym")


def kfac_pack_sym_static(ms: Sequence, packed, direction: int, stream=None) -> None:
    """kfac_pack_sym without a workspace: the library's own device array holds
    the layer table, and nothing is allocated (at most 1024 factors; calls
    that may overlap on one GPU race)."""
    import torch
    lib = load_library()
    dev = _check(list(ms) + [packed], torch.float32, "kfac_pack_sym_static")
    d = []
    for m in ms:
        if m.dim() != 2 or m.shape[0] != m.shape[1]:
            raise ValueError("kfac_pack_sym_static: factors must be square")
        d.append(m.shape[0])
    if packed.numel() != kfac_packed_size(d):
        raise ValueError("kfac_pack_sym_static: packed buffer has the wrong length")
    _call(lib.kfac_pack_sym_static(len(ms), _ptrs(ms), _i64(d), ctypes.c_void_p(packed.data_ptr()), int(direction),
                                   _stream(dev, stream)), "kfac_pack_sym_static")


def kfac_stream_copy(src, dst, stream=None) -> None:
    """dst <- src, a plain device copy (the streaming reference of pack)."""
    lib = load_library()
    dev = _check([src, dst], None, "kfac_stream_copy")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("kfac_stream_copy: source and destination sizes differ")
    _call(lib.kfac_stream_copy(ctypes.c_void_p(src.data_ptr()), ctypes.c_void_p(dst.data_ptr()), nbytes,
                               _stream(dev, stream)), "kfac_stream_copy")


KFAC_RATE_BF16, KFAC_RATE_F64, KFAC_RATE_F32 = 0, 1, 2


def kfac_matrix_rate(kind: int, iters: int, sink, stream=None) -> float:
    """Register-only matrix-core product loops (the measured reference of the
    matrix-core-bound stages); sink float32 with 4 entries per workgroup.
    Returns the flops the call runs."""
    import torch
    lib = load_library()
    dev = _check([sink], torch.float32, "kfac_matrix_rate")
    if sink.numel() % 4 != 0 or sink.numel() == 0:
        raise ValueError("kfac_matrix_rate: sink needs 4 floats per workgroup")
    flops = ctypes.c_double(0.0)
    _call(lib.kfac_matrix_rate(int(kind), int(iters), sink.numel() // 4, ctypes.c_void_p(sink.data_ptr()),
                               ctypes.byref(flops), _stream(dev, stream)), "kfac_matrix_rate")
    return flops.value


def kfac_damped_inverse(xs: Sequence, gamma: float, xinvs: Sequence, info, stream=None) -> None:
    """xinv_i <- (X_i + gamma I)^-1 (X_i read from the upper triangle), info int32 [n]."""
    import torch
    lib = load_library()
    if len(xs) != len(xinvs) or len(xs) == 0:
        raise ValueError("kfac_damped_inverse: need equally many inputs and outputs")
    dev = _check(list(xs) + list(xinvs), torch.float32, "kfac_damped_inverse")
    _check([info], torch.int32, "kfac_damped_inverse(info)")
    if info.numel() != len(xs):
        raise ValueError("kfac_damped_inverse: info needs one entry per matrix")
    d = []
    for x, z in zip(xs, xinvs):
        if x.dim() != 2 or x.shape[0] != x.shape[1] or z.shape != x.shape:
            raise ValueError("kfac_damped_inverse: square inputs and outputs of equal shape")
        d.append(x.shape[0])
    n = len(xs)
    d64 = _i64(d)
    with _on(stream):
        ws = _workspace(lib.kfac_inverse_workspace_size(n, d64), dev)
    _call(lib.kfac_damped_inverse(n, _ptrs(xs), d64, ctypes.c_float(gamma), _ptrs(xinvs),
                                  ctypes.c_void_p(info.data_ptr()), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                                  _stream(dev, stream)), "kfac_damped_inverse")


def kfac_precondition(ginvs: Sequence, grads: Sequence, ainvs: Sequence, outs: Sequence, stream=None) -> None:
    """out_l <- ginv_l . grad_l . ainv_l (ginv, ainv symmetric)."""
    import torch
    lib = load_library()
    n = len(grads)
    if not (len(ginvs) == len(ainvs) == len(outs) == n) or n == 0:
        raise ValueError("kfac_precondition: need equally many of every argument")
    dev = _check(list(ginvs) + list(grads) + list(ainvs) + list(outs), torch.float32, "kfac_precondition")
    dg, da = [], []
    for zg, g, za, o in zip(ginvs, grads, ainvs, outs):
        if g.dim() != 2 or zg.shape != (g.shape[0], g.shape[0]) or za.shape != (g.shape[1], g.shape[1]) \
                or o.shape != g.shape:
            raise ValueError("kfac_precondition: shapes must be ginv [dg,dg], grad [dg,da], ainv [da,da], out [dg,da]")
        dg.append(g.shape[0])
        da.append(g.shape[1])
    g64, a64 = _i64(dg), _i64(da)
    with _on(stream):
        ws = _workspace(lib.kfac_precondition_workspace_size(n, g64, a64), dev)
    _call(lib.kfac_precondition(n, _ptrs(ginvs), _ptrs(grads), _ptrs(ainvs), g64, a64, _ptrs(outs),
                                ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(dev, stream)),
          "kfac_precondition")


__all__ = [
    "load_library", "status_string", "KfacError", "KfacLibraryError",
    "kfac_factors", "kfac_packed_size", "kfac_pack_sym", "kfac_pack_sym_static", "kfac_stream_copy",
    "kfac_matrix_rate", "KFAC_RATE_BF16", "KFAC_RATE_F64", "KFAC_RATE_F32",
    "kfac_damped_inverse",
    "kfac_precondition",
    "kfac_attention_forward", "kfac_attention_backward", "kfac_position_borders",
    "kfac_checkpoint_empty", "kfac_checkpoint_store", "kfac_checkpoint_load", "kfac_checkpoint_factors",
    "kfac_checkpoint_grad",
    "kfac_layer_norm_forward", "kfac_layer_norm_backward", "kfac_gated_forward", "kfac_gated_backward", "KFAC_ACTIVATIONS",
    "kfac_grad_norm", "kfac_grad_clip",
    "KFAC_F32", "KFAC_BF16", "KFAC_PACK", "KFAC_UNPACK", "KFAC_MAX_COUNT", "EXPORTS",
]


def conv_out_hw(h: int, w: int, kh: int, kw: int, stride=(1, 1), padding=(0, 0), dilation=(1, 1)):
    """Output height and width of a convolution (the formula of kfac_im2col)."""
    oh = (h + 2 * padding[0] - dilation[0] * (kh - 1) - 1) // stride[0] + 1
    ow = (w + 2 * padding[1] - dilation[1] * (kw - 1) - 1) // stride[1] + 1
    return oh, ow


def kfac_im2col(xs: Sequence, shapes: Sequence[dict], outs: Sequence, stream=None) -> None:
    """a = patches of x as rows (kfac_im2col).  xs[i]: [n, c, h, w] float32 or
    bfloat16; shapes[i]: dict with kh, kw, stride, padding, dilation, ones;
    outs[i]: [n*oh*ow, c*kh*kw + ones] of the same dtype."""
    import torch
    lib = load_library()
    if len(xs) != len(shapes) or len(xs) != len(outs) or len(xs) == 0:
        raise ValueError("kfac_im2col: need equally many inputs, shapes and outputs")
    dt = xs[0].dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("kfac_im2col: inputs must be float32 or bfloat16")
    dev = _check(list(xs) + list(outs), dt, "kfac_im2col")
    n = len(xs)
    arr = (KfacConv * n)()
    for i, (x, sh, o) in enumerate(zip(xs, shapes, outs)):
        if x.dim() != 4:
            raise ValueError("kfac_im2col: inputs must be [n, c, h, w]")
        kh, kw = sh.get("kernel", (1, 1))
        st, pd, dl = sh.get("stride", (1, 1)), sh.get("padding", (0, 0)), sh.get("dilation", (1, 1))
        ones = int(bool(sh.get("ones", False)))
        oh, ow = conv_out_hw(x.shape[2], x.shape[3], kh, kw, st, pd, dl)
        if o.dim() != 2 or o.shape != (x.shape[0] * oh * ow, x.shape[1] * kh * kw + ones):
            raise ValueError("kfac_im2col: output has the wrong shape")
        arr[i] = KfacConv(x.shape[0], x.shape[1], x.shape[2], x.shape[3], kh, kw, st[0], st[1], pd[0], pd[1],
                          dl[0], dl[1], ones, 0)
    with _on(stream):
        ws = _workspace(lib.kfac_im2col_workspace_size(n), dev)
    dtype = KFAC_BF16 if dt == torch.bfloat16 else KFAC_F32
    _call(lib.kfac_im2col(n, _ptrs(xs), ctypes.cast(arr, ctypes.c_void_p), dtype, _ptrs(outs),
                          ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(dev, stream)), "kfac_im2col")


def kfac_grad_rows(gys: Sequence, scale: float, outs: Sequence, stream=None) -> None:
    """g[b*hw + p][c] = scale * gy[b][c][p] (kfac_grad_rows).  gys[i]:
    [b, c] or [b, c, H, W], float32 or bfloat16; outs[i]: [b*H*W, c]."""
    import torch
    lib = load_library()
    if len(gys) != len(outs) or len(gys) == 0:
        raise ValueError("kfac_grad_rows: need equally many gradients and outputs")
    dt = gys[0].dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError("kfac_grad_rows: gradients must be float32 or bfloat16")
    dev = _check(list(gys) + list(outs), dt, "kfac_grad_rows")
    b, c, hw = [], [], []
    for gy, o in zip(gys, outs):
        if gy.dim() < 2:
            raise ValueError("kfac_grad_rows: gradients must be [b, c, ...]")
        p = 1
        for s_ in gy.shape[2:]:
            p *= s_
        if o.shape != (gy.shape[0] * p, gy.shape[1]):
            raise ValueError("kfac_grad_rows: output has the wrong shape")
        b.append(gy.shape[0]); c.append(gy.shape[1]); hw.append(p)
    n = len(gys)
    with _on(stream):
        ws = _workspace(lib.kfac_grad_rows_workspace_size(n), dev)
    dtype = KFAC_BF16 if dt == torch.bfloat16 else KFAC_F32
    _call(lib.kfac_grad_rows(n, _ptrs(gys), _i64(b), _i64(c), _i64(hw), dtype, ctypes.c_float(scale), _ptrs(outs),
                             ctypes.c_void_p(ws.data_ptr()), ws.numel(), _stream(dev, stream)), "kfac_grad_rows")


def kfac_grad_matrix(wgrads: Sequence, bgrads: Sequence, mats: Sequence, direction: int, stream=None) -> None:
    """KFAC_PACK: mats[i] = [wgrad | bgrad]; KFAC_UNPACK: the reverse.
    wgrads[i]: float32 with d_out = shape[0] and d_in = the rest flattened;
    bgrads[i]: [d_out] or None; mats[i]: [d_out, d_in + has_bias]."""
    import torch
    lib = load_library()
    if len(wgrads) != len(bgrads) or len(wgrads) != len(mats) or len(wgrads) == 0:
        raise ValueError("kfac_grad_matrix: need equally many weights, biases and matrices")
    dev = _check(list(wgrads) + [b for b in bgrads if b is not None] + list(mats), torch.float32, "kfac_grad_matrix")
    d_out, d_in = [], []
    for w, b, m in zip(wgrads, bgrads, mats):
        do = w.shape[0]
        di = w.numel() // do
        if b is not None and b.numel() != do:
            raise ValueError("kfac_grad_matrix: bias gradient has the wrong length")
        if m.shape != (do, di + (b is not None)):
            raise ValueError("kfac_grad_matrix: matrix has the wrong shape")
        d_out.append(do); d_in.append(di)
    n = len(wgrads)
    bptr = (ctypes.c_void_p * n)(*[b.data_ptr() if b is not None else None for b in bgrads])
    with _on(stream):
        ws = _workspace(lib.kfac_grad_matrix_workspace_size(n), dev)
    _call(lib.kfac_grad_matrix(n, _ptrs(wgrads), ctypes.cast(bptr, ctypes.c_void_p), _i64(d_out), _i64(d_in),
                               _ptrs(mats), int(direction), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
                               _stream(dev, stream)), "kfac_grad_matrix")


# --------------------------------------------------------------- attention --

def kfac_position_borders(buckets: int, max_distance: int) -> list:
    """Distances at which the buckets of one side begin, the first (at 0) left
    out: the first half of the buckets hold one distance each, the others
    widen with the logarithm, the last one beginning at the least distance t
    with (t / h)^w >= (max_distance / h)^(w - 1), h and w the counts of narrow
    and wide buckets.  Whole-number arithmetic."""
    buckets, max_distance = int(buckets), int(max_distance)
    if buckets < 1:
        raise ValueError("kfac_position_borders: at least one bucket")
    near = buckets // 2
    wide = buckets - near
    if near == 0:
        return []
    if max_distance <= near:
        raise ValueError("kfac_position_borders: max_distance must exceed the narrow buckets' distances")
    borders = list(range(1, near + 1))
    for m in range(1, wide):
        lo, hi = borders[-1], max_distance
        goal = max_distance ** m * near ** (wide - m)
        while lo < hi:                      # the least t with t^wide >= max_distance^m near^(wide - m)
            mid = (lo + hi) // 2
            if mid ** wide >= goal:
                hi = mid
            else:
                lo = mid + 1
        borders.append(max(lo, borders[-1] + 1))
    return borders


def _heads(t, shape, dtype, device, name) -> bytes:
    """kfac_tensor4_t of a [batch, rows, heads, dim] tensor, dim contiguous."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected torch tensors")
    if t.get_device() != device:
        raise ValueError(f"{name}: tensors must live on the GPU, all on one device")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shapes must be q, out, dout, dq [batch, len_q, heads, dim], "
                         f"k, v, dk, dv [batch, len_k, kv_heads, dim]; got {tuple(t.shape)} for {tuple(shape)}")
    sb, sl, sh, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return _TENSOR4.pack(t.data_ptr(), sb, sl, sh)


def _attention_form(name, q, k, v, lse, scale, causal, lens, bias, borders, two_sided):
    """kfac_attention_t of a call, its dtype, the packed q, k, v and the host
    array that the form points to."""
    import torch
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor):
        raise TypeError(f"{name}: expected torch tensors")
    dt = q.dtype
    if dt is torch.bfloat16:
        dtype = KFAC_BF16
    elif dt is torch.float32:
        dtype = KFAC_F32
    else:
        raise ValueError(f"{name}: tensors must be float32 or bfloat16")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"{name}: expected [batch, rows, heads, dim]")
    if not q.is_cuda:
        raise ValueError(f"{name}: tensors must live on the GPU")
    dev = q.get_device()
    b, lq, h, d = q.shape
    kb, lk, hk, kd = shape = k.shape
    if kb != b or kd != d:
        raise ValueError(f"{name}: shapes must be q [batch, len_q, heads, dim], k and v [batch, len_k, kv_heads, dim]")
    packed = (_heads(q, q.shape, dt, dev, name), _heads(k, shape, dt, dev, name), _heads(v, shape, dt, dev, name))
    _flat(lse, (b, h, lq), torch.float32, dev, f"{name}(lse)")
    at, n, at_ptr, bias_ptr, lens_ptr = None, 0, 0, 0, 0
    if lens is not None:
        lens_ptr = _flat(lens, (b,), torch.int32, dev, f"{name}(lens)")
    if bias is not None:
        n = len(borders) if borders is not None else 0
        bias_ptr = _flat(bias, ((n + 1) * (2 if two_sided else 1), h), torch.float32, dev, f"{name}(bias)")
        if n:
            try:
                at = struct.pack(f"@{n}i", *borders)
            except struct.error:
                raise ValueError(f"{name}: borders must be whole numbers below 2^31") from None
            at_ptr = ctypes.cast(at, ctypes.c_void_p).value
    elif borders is not None and len(borders):
        raise ValueError(f"{name}: borders without a bias")
    form = _ATTENTION.pack(b, lq, lk, h, hk, d, 1 if causal else 0, d ** -0.5 if scale is None else scale, n,
                           1 if two_sided else 0, at_ptr, lens_ptr, bias_ptr)
    return form, dtype, packed, dev, at


def _flat(t, shape, dtype, device, name) -> int:
    """Address of a contiguous tensor of the given shape."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected torch tensors")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: tensors must live on the GPU, all on one device")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    return t.data_ptr()


def _space(need, device, name):
    """Workspace of a call: (tensor or None, address, bytes)."""
    import torch
    if need == 0:
        return None, 0, 0
    if need == ctypes.c_size_t(-1).value:
        raise KfacError(KFAC_ERR_INVALID_VALUE, name)
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), need


def kfac_attention_forward(q, k, v, out, lse, scale=None, causal=False, lens=None, bias=None, borders=None,
                           two_sided=True, stream=None) -> None:
    """out, lse <- attention of q [batch, len_q, heads, dim] over k, v [batch,
    len_k, kv_heads, dim] (float32 or bfloat16; out like q, lse float32
    [batch, heads, len_q]).  scale: 1 / sqrt(dim) by default.  lens: int32
    [batch], keys visible per sequence.  bias: float32 [buckets, heads] with
    ascending `borders` of the buckets (see kfac_position_borders)."""
    lib = load_library()
    name = "kfac_attention_forward"
    form, dtype, (tq, tk, tv), dev, at = _attention_form(name, q, k, v, lse, scale, causal, lens, bias, borders, two_sided)
    to = _heads(out, q.shape, q.dtype, dev, name)
    with _on(stream):
        ws, at_ws, size = _space(lib.kfac_attention_workspace_size(form, dtype, 0), q.device, name)
    _call(lib.kfac_attention_forward(form, dtype, tq, tk, tv, to, lse.data_ptr(), at_ws, size, _stream(q.device, stream)),
          name)


def kfac_attention_backward(q, k, v, out, lse, dout, dq, dk, dv, dbias=None, scale=None, causal=False, lens=None,
                            bias=None, borders=None, two_sided=True, stream=None) -> None:
    """dq, dk, dv (shaped like q, k, v) and dbias (like bias) <- gradients of
    kfac_attention_forward, from its inputs, out, lse and the gradient dout."""
    import torch
    lib = load_library()
    name = "kfac_attention_backward"
    form, dtype, (tq, tk, tv), dev, at = _attention_form(name, q, k, v, lse, scale, causal, lens, bias, borders, two_sided)
    dt, rows, keys = q.dtype, q.shape, k.shape
    if (bias is None) != (dbias is None):
        raise ValueError(f"{name}: bias and dbias come together")
    at_dbias = 0 if dbias is None else _flat(dbias, bias.shape, torch.float32, dev, f"{name}(dbias)")
    to, tdo, tdq = (_heads(t, rows, dt, dev, name) for t in (out, dout, dq))
    tdk, tdv = (_heads(t, keys, dt, dev, name) for t in (dk, dv))
    with _on(stream):
        ws, at_ws, size = _space(lib.kfac_attention_workspace_size(form, dtype, 1), q.device, name)
    _call(lib.kfac_attention_backward(form, dtype, tq, tk, tv, to, lse.data_ptr(), tdo, tdq, tdk, tdv, at_dbias, at_ws, size,
                                      _stream(q.device, stream)), name)


# ------------------------------------------------------------- checkpoints --

KEEP_BLOCK = 32


def kfac_checkpoint_empty(rows: int, d: int, device):
    """Room for a checkpoint of [rows, d] (d with the column of ones): codes
    uint8 [ceil(rows / 32), d, 32] and scales uint8 [ceil(rows / 32), d]."""
    import torch
    blocks = (int(rows) + KEEP_BLOCK - 1) // KEEP_BLOCK
    return (torch.empty(blocks, int(d), KEEP_BLOCK, dtype=torch.uint8, device=device),
            torch.empty(blocks, int(d), dtype=torch.uint8, device=device))


def _pack_i64(values) -> bytes:
    try:
        return struct.pack(f"@{len(values)}q", *values)
    except struct.error:
        raise ValueError("sizes must be whole numbers") from None


def _pack_ptrs(values) -> bytes:
    return struct.pack(f"@{len(values)}P", *values)


def _kept(codes, scales, rows, name):
    """The checkpoints of a call, whose rows come from the matrices that go
    with them: packed addresses of codes and scales and packed rows, columns,
    device index and device."""
    import torch
    n = len(codes)
    if n == 0 or n != len(scales) or n != len(rows):
        raise ValueError(f"{name}: need equally many of every argument")
    at_c, at_s, d, index, u8 = [], [], [], None, torch.uint8
    for c, s, r in zip(codes, scales, rows):
        if not isinstance(c, torch.Tensor) or not isinstance(s, torch.Tensor):
            raise TypeError(f"{name}: expected torch tensors")
        where = c.get_device()
        if index is None:
            index = where
        if where < 0 or where != index or s.get_device() != index:
            raise ValueError(f"{name}: tensors must live on the GPU, all on one device")
        shape = c.shape
        if c.dtype is not u8 or s.dtype is not u8 or len(shape) != 3 or shape[2] != KEEP_BLOCK \
                or shape[0] != (r + KEEP_BLOCK - 1) // KEEP_BLOCK or s.shape != shape[:2]:
            raise ValueError(f"{name}: codes must be uint8 [ceil(rows / 32), d, 32] and scales [ceil(rows / 32), d]")
        if not c.is_contiguous() or not s.is_contiguous():
            raise ValueError(f"{name}: tensors must be contiguous")
        at_c.append(c.data_ptr())
        at_s.append(s.data_ptr())
        d.append(shape[1])
    return _pack_ptrs(at_c), _pack_ptrs(at_s), _pack_i64(rows), d, index, codes[0].device


def _matrices(ts, index, name):
    """Addresses, rows, columns and the common library type of contiguous
    two-dimensional matrices on one device (None: the first one's)."""
    import torch
    if not ts:
        raise ValueError(f"{name}: need equally many of every argument")
    at, rows, cols, dt = [], [], [], None
    for t in ts:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}: expected torch tensors")
        shape = t.shape
        if len(shape) != 2:
            raise ValueError(f"{name}: matrices must be two-dimensional")
        if dt is None:
            dt = t.dtype
            if dt is not torch.bfloat16 and dt is not torch.float32:
                raise ValueError(f"{name}: matrices must be float32 or bfloat16")
        elif t.dtype is not dt:
            raise ValueError(f"{name}: expected {dt}, got {t.dtype}")
        where = t.get_device()
        if index is None:
            index = where
        if where < 0 or where != index:
            raise ValueError(f"{name}: tensors must live on the GPU, all on one device")
        if not t.is_contiguous():
            raise ValueError(f"{name}: tensors must be contiguous")
        at.append(t.data_ptr())
        rows.append(shape[0])
        cols.append(shape[1])
    return _pack_ptrs(at), rows, cols, KFAC_BF16 if dt is torch.bfloat16 else KFAC_F32, index


def kfac_checkpoint_store(xs: Sequence, codes: Sequence, scales: Sequence, ones: bool = False, stream=None) -> None:
    """codes_i, scales_i <- x_i [rows, d] in 8 bits (see kfac_checkpoint_empty;
    d + 1 columns with `ones`, the last one all ones)."""
    lib = load_library()
    name = "kfac_checkpoint_store"
    if not len(xs) == len(codes) == len(scales):
        raise ValueError(f"{name}: need equally many of every argument")
    at, rows, cols, dtype, index = _matrices(xs, None, name)
    ones = 1 if ones else 0
    at_c, at_s, r64, d, where, device = _kept(codes, scales, rows, name)
    if where != index:
        raise ValueError(f"{name}: all tensors must be on one device")
    if d != ([c + 1 for c in cols] if ones else cols):
        raise ValueError(f"{name}: checkpoints must hold the input's columns" + (" and the column of ones" if ones else ""))
    _call(lib.kfac_checkpoint_store(len(d), at, r64, _pack_i64(cols), ones, dtype, at_c, at_s, _stream(device, stream)),
          name)


def kfac_checkpoint_load(codes: Sequence, scales: Sequence, ys: Sequence, stream=None) -> None:
    """y_i [rows, cols] float32 or bfloat16 <- the first cols columns of what checkpoint i stands for."""
    lib = load_library()
    name = "kfac_checkpoint_load"
    if not len(ys) == len(codes) == len(scales):
        raise ValueError(f"{name}: need equally many of every argument")
    at, rows, cols, dtype, index = _matrices(ys, None, name)
    at_c, at_s, r64, d, where, device = _kept(codes, scales, rows, name)
    if where != index:
        raise ValueError(f"{name}: all tensors must be on one device")
    if any(c > n for c, n in zip(cols, d)):
        raise ValueError(f"{name}: more columns than the checkpoint holds")
    _call(lib.kfac_checkpoint_load(len(d), at_c, at_s, r64, _pack_i64(d), _pack_i64(cols), dtype, at,
                                   _stream(device, stream)), name)


def kfac_checkpoint_factors(codes: Sequence, scales: Sequence, rows: Sequence, ms: Sequence, eps: float,
                            first_step: bool, stream=None) -> None:
    """kfac_factors of kept inputs: M_i <- F_i (first step) or eps*M_i +
    (1-eps)*F_i, F_i = x_i^T x_i / rows_i, upper triangle of each float32 M_i."""
    import torch
    lib = load_library()
    name = "kfac_checkpoint_factors"
    if len(ms) != len(codes):
        raise ValueError(f"{name}: need equally many checkpoints and factors")
    at_c, at_s, r64, d, index, device = _kept(codes, scales, rows, name)
    at = _pack_ptrs([_flat(m, (n, n), torch.float32, index, f"{name}(m)") for m, n in zip(ms, d)])
    n, d64 = len(d), _pack_i64(d)
    with _on(stream):
        ws, at_ws, size = _space(lib.kfac_checkpoint_factors_workspace_size(n, r64, d64), device, name)
    _call(lib.kfac_checkpoint_factors(n, at_c, at_s, r64, d64, at, eps, 1 if first_step else 0, at_ws, size,
                                      _stream(device, stream)), name)


def kfac_checkpoint_grad(gs: Sequence, codes: Sequence, scales: Sequence, mats: Sequence, stream=None) -> None:
    """mat_i [d_out, d] float32 <- g_i^T x_i from a kept input: the weight
    gradient, with the bias gradient in the last column where the checkpoint
    has a column of ones; g_i [rows, d_out] float32 or bfloat16."""
    import torch
    lib = load_library()
    name = "kfac_checkpoint_grad"
    if len(mats) != len(gs):
        raise ValueError(f"{name}: need equally many gradients and matrices")
    at, rows, d_out, dtype, index = _matrices(gs, None, name)
    at_c, at_s, r64, d, where, device = _kept(codes, scales, rows, name)
    if where != index:
        raise ValueError(f"{name}: all tensors must be on one device")
    out = _pack_ptrs([_flat(m, (o, n), torch.float32, index, f"{name}(mat)") for m, o, n in zip(mats, d_out, d)])
    n, o64, d64 = len(d), _pack_i64(d_out), _pack_i64(d)
    with _on(stream):
        ws, at_ws, size = _space(lib.kfac_checkpoint_grad_workspace_size(n, r64, o64, d64), device, name)
    _call(lib.kfac_checkpoint_grad(n, at, at_c, at_s, r64, o64, d64, dtype, out, at_ws, size, _stream(device, stream)),
          name)


# -------------------------------------------------------------- layer norm --

def _elsewhere(index):
    """Whether a device is not the current one (a call's launches go to the current one)."""
    import torch
    return torch._C._cuda_getDevice() != index


def _raw_stream(index, stream):
    """Handle of the given stream, or of the device's current one."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _type_of(t, name):
    """Library type and torch type of a call's tensors, by one of them."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected torch tensors")
    dt = t.dtype
    if dt is torch.bfloat16:
        return KFAC_BF16, dt
    if dt is torch.float32:
        return KFAC_F32, dt
    raise ValueError(f"{name}: tensors must be float32 or bfloat16")


def _row_matrix(t, shape, dtype, device, name):
    """Address and row stride of a matrix whose rows are contiguous."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected torch tensors")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: tensors must live on the GPU, all on one device")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")
    row, col = t.stride()
    if col != 1 and shape[1] > 1 and shape[0]:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), row


def _norm_rows(x, name):
    """Library type, torch type, shape, device index, address and row stride of a call's rows."""
    dtype, dt = _type_of(x, name)
    dev, shape = x.get_device(), x.shape
    if len(shape) != 2 or dev < 0:
        raise ValueError(f"{name}: expected a matrix [rows, d] on the GPU")
    row, col = x.stride()
    if col != 1 and shape[1] > 1 and shape[0]:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return dtype, dt, shape, dev, x.data_ptr(), row


def _norm_vectors(vectors, shape, dtype, device, name):
    """The vectors' common library type (that of the rows where there is none) and their addresses."""
    import torch
    kind, at = None, []
    for t in vectors:
        if t is None:
            at.append(None)
            continue
        if kind is None:
            kind = t.dtype if isinstance(t, torch.Tensor) else None
            if kind is not torch.float32 and kind is not dtype:
                raise ValueError(f"{name}: weight, bias and their gradients must be float32 or of the rows' type, all alike")
        at.append(_flat(t, shape, kind, device, name))
    return KFAC_BF16 if (kind or dtype) is torch.bfloat16 else KFAC_F32, at


def kfac_layer_norm_forward(x, y, mean=None, rstd=None, weight=None, bias=None, eps=1e-5, stream=None) -> None:
    """y <- weight (x - mean) rstd + bias over each row of x [rows, d]
    (float32 or bfloat16, rows contiguous, any stride between them; y alike),
    rstd = 1 / sqrt(variance + eps).  mean, rstd: float32 [rows], for the
    backward pass, or None; weight, bias: [d], float32 or of x's type, or None."""
    import torch
    lib = load_library()
    name = "kfac_layer_norm_forward"
    dtype, dt, shape, dev, at_x, sx = _norm_rows(x, name)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return kfac_layer_norm_forward(x, y, mean, rstd, weight, bias, eps, stream)
    at_y, sy = _row_matrix(y, shape, dt, dev, name)
    at_m = None if mean is None else _flat(mean, shape[:1], torch.float32, dev, name)
    at_r = None if rstd is None else _flat(rstd, shape[:1], torch.float32, dev, name)
    kind, (at_w, at_b) = _norm_vectors((weight, bias), shape[1:], dt, dev, name)
    _call(lib.kfac_layer_norm_forward(shape[0], shape[1], dtype, at_x, sx, at_y, sy, at_m, at_r, at_w, at_b, kind, eps,
                                      _raw_stream(dev, stream)), name)


def kfac_layer_norm_backward(dy, x, mean, rstd, dx=None, weight=None, dweight=None, dbias=None, stream=None) -> None:
    """dx (like x), dweight and dbias [d] <- gradients of
    kfac_layer_norm_forward from the output's gradient dy (like x), its input
    and its statistics; an output that is None is not formed."""
    import torch
    lib = load_library()
    name = "kfac_layer_norm_backward"
    dtype, dt, shape, dev, at_x, sx = _norm_rows(x, name)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return kfac_layer_norm_backward(dy, x, mean, rstd, dx, weight, dweight, dbias, stream)
    at_dy, sdy = _row_matrix(dy, shape, dt, dev, name)
    at_dx, sdx = (None, shape[1]) if dx is None else _row_matrix(dx, shape, dt, dev, name)
    at_m = _flat(mean, shape[:1], torch.float32, dev, name)
    at_r = _flat(rstd, shape[:1], torch.float32, dev, name)
    kind, (at_w, at_dw, at_db) = _norm_vectors((weight, dweight, dbias), shape[1:], dt, dev, name)
    ws, at_ws, size = None, None, 0
    if dweight is not None or dbias is not None:
        with _on(stream):
            ws, at_ws, size = _space(lib.kfac_layer_norm_workspace_size(shape[0], shape[1]), x.device, name)
    _call(lib.kfac_layer_norm_backward(shape[0], shape[1], dtype, at_dy, sdy, at_x, sx, at_m, at_r, at_w, at_dx, sdx, at_dw,
                                       at_db, kind, at_ws, size, _raw_stream(dev, stream)), name)


# ------------------------------------------------------------------- gated --

KFAC_ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}


def _gated_call(name, x, weight, activation):
    """Sizes (rows, d, width), types, device index, activation and x's address."""
    import torch
    dtype, dt = _type_of(x, name)
    if not isinstance(weight, torch.Tensor):
        raise TypeError(f"{name}: expected torch tensors")
    dev, shape, wide = x.get_device(), x.shape, weight.shape
    if len(shape) != 2 or len(wide) != 2 or dev < 0:
        raise ValueError(f"{name}: expected matrices x [rows, d] and weight [2 width, d] on the GPU")
    if wide[0] % 2:
        raise ValueError(f"{name}: weight must hold as many rows for the gate as for the other projection")
    act = KFAC_ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"{name}: activation must be one of {', '.join(KFAC_ACTIVATIONS)}")
    rows, d = shape
    return rows, d, wide[0] // 2, dtype, dt, dev, act


def kfac_gated_forward(x, weight, h, bias=None, pre=None, activation="silu", stream=None) -> None:
    """h [rows, width] <- act(g) u with [g | u] = x weight^T + bias, x [rows, d],
    weight [2 width, d] with the gate's rows first (all float32 or all
    bfloat16), bias [2 width] float32.  pre [rows, 2 width] <- [g | u], which the
    backward pass needs."""
    import torch
    lib = load_library()
    name = "kfac_gated_forward"
    rows, d, width, dtype, dt, dev, act = _gated_call(name, x, weight, activation)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return kfac_gated_forward(x, weight, h, bias, pre, activation, stream)
    at_x = _flat(x, (rows, d), dt, dev, f"{name}(x)")
    at_w = _flat(weight, (2 * width, d), dt, dev, f"{name}(weight)")
    at_h = _flat(h, (rows, width), dt, dev, f"{name}(h)")
    at_b = None if bias is None else _flat(bias, (2 * width,), torch.float32, dev, f"{name}(bias)")
    at_pre = None if pre is None else _flat(pre, (rows, 2 * width), dt, dev, f"{name}(pre)")
    need = lib.kfac_gated_workspace_size(rows, d, width, dtype, 0)
    ws, at_ws, size = None, None, 0
    if need:
        with _on(stream):
            ws, at_ws, size = _space(need, x.device, name)
    _call(lib.kfac_gated_forward(rows, d, width, dtype, act, at_x, at_w, at_b, at_h, at_pre, at_ws, size,
                                 _raw_stream(dev, stream)), name)


def kfac_gated_backward(dh, x, weight, pre, dpre, dx=None, dweight=None, dbias=None, activation="silu", stream=None) -> None:
    """dpre [rows, 2 width], dx (like x), dweight (like weight, or float32) and
    dbias [2 width] float32 <- gradients of kfac_gated_forward from the output's
    gradient dh [rows, width], its inputs and pre; an output that is None is
    not formed.  dpre is like x, or float32 beside bfloat16: dx and dweight are
    formed from it as it is given out, so that only a bfloat16 dpre is rounded
    before them (and is a third of the work)."""
    import torch
    lib = load_library()
    name = "kfac_gated_backward"
    rows, d, width, dtype, dt, dev, act = _gated_call(name, x, weight, activation)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return kfac_gated_backward(dh, x, weight, pre, dpre, dx, dweight, dbias, activation, stream)
    wide = (rows, 2 * width)
    at_dh = _flat(dh, (rows, width), dt, dev, f"{name}(dh)")
    at_x = _flat(x, (rows, d), dt, dev, f"{name}(x)")
    at_w = _flat(weight, (2 * width, d), dt, dev, f"{name}(weight)")
    at_pre = _flat(pre, wide, dt, dev, f"{name}(pre)")
    unrounded = dtype == KFAC_BF16 and _type_of(dpre, f"{name}(dpre)")[0] == KFAC_F32
    at_dpre = _flat(dpre, wide, torch.float32 if unrounded else dt, dev, f"{name}(dpre)")
    at_dx = None if dx is None else _flat(dx, (rows, d), dt, dev, f"{name}(dx)")
    at_dw, kind = None, KFAC_F32
    if dweight is not None:
        kind, kept = _type_of(dweight, f"{name}(dweight)")
        at_dw = _flat(dweight, (2 * width, d), kept, dev, f"{name}(dweight)")
    at_db = None if dbias is None else _flat(dbias, (2 * width,), torch.float32, dev, f"{name}(dbias)")
    with _on(stream):
        ws, at_ws, size = _space(lib.kfac_gated_workspace_size(rows, d, width, dtype, 2 if unrounded else 1), x.device, name)
    rest = at_dh, at_x, at_w, at_pre, at_dpre, at_dx, at_dw, kind, at_db, at_ws, size, _raw_stream(dev, stream)
    if unrounded:
        _call(lib.kfac_gated_backward_f32(rows, d, width, act, *rest), name)
    else:
        _call(lib.kfac_gated_backward(rows, d, width, dtype, act, *rest), name)


# ----------------------------------------------------------- gradient norm --

KFAC_MAX_COUNT = 4096   # gradients of a call


def _gradients(ts, name):
    """Addresses, element counts and torch types of contiguous tensors of any
    shape on one device, and the device's index.  (Each property in one
    pass over all of them: a model has hundreds of gradients.)"""
    import torch
    cls = torch.Tensor
    if len(ts) == 0:
        raise ValueError(f"{name}: need at least one gradient")
    if len(ts) > KFAC_MAX_COUNT:
        raise ValueError(f"{name}: {len(ts)} gradients, a call takes at most {KFAC_MAX_COUNT}")
    try:
        where = set(map(cls.get_device, ts))
    except TypeError:
        raise TypeError(f"{name}: expected torch tensors") from None
    index = where.pop()
    if where or index < 0:
        raise ValueError(f"{name}: tensors must live on the GPU, all on one device")
    if not all(map(cls.is_contiguous, ts)):
        raise ValueError(f"{name}: tensors must be contiguous")
    kinds = list(map(cls.dtype.__get__, ts))
    if not {torch.float32, torch.bfloat16}.issuperset(kinds):
        raise ValueError(f"{name}: tensors must be float32 or bfloat16")
    return list(map(cls.data_ptr, ts)), list(map(cls.numel, ts)), kinds, index


def _pack_kinds(kinds) -> bytes:
    import torch
    bf16 = torch.bfloat16
    return struct.pack(f"@{len(kinds)}i", *[KFAC_BF16 if k is bf16 else KFAC_F32 for k in kinds])


def kfac_grad_norm(grads: Sequence, norm, stream=None) -> None:
    """norm [1] float32 <- the square root of the sum of all squares of the
    gradients (float32 or bfloat16, contiguous, of any shapes; at most 4096)."""
    import torch
    lib = load_library()
    name = "kfac_grad_norm"
    at, count, kinds, dev = _gradients(grads, name)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return kfac_grad_norm(grads, norm, stream)
    at_norm = _flat(norm, (1,), torch.float32, dev, f"{name}(norm)")
    n = len(count)
    with _on(stream):
        ws, at_ws, size = _space(lib.kfac_grad_norm_workspace_size(n), norm.device, name)
    _call(lib.kfac_grad_norm(n, _pack_ptrs(at), _pack_i64(count), _pack_kinds(kinds), at_norm, at_ws, size,
                             _raw_stream(dev, stream)), name)


def kfac_grad_clip(grads: Sequence, max_norm: float, norm, outs: Sequence = None, stream=None) -> None:
    """norm <- as kfac_grad_norm; out_i <- min(1, max_norm / (norm + 1e-6))
    grad_i, in place where `outs` is None.  No two of the tensors may overlap,
    apart from an out that is its gradient itself."""
    import torch
    lib = load_library()
    name = "kfac_grad_clip"
    at, count, kinds, dev = _gradients(grads, name)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return kfac_grad_clip(grads, max_norm, norm, outs, stream)
    at_norm = _flat(norm, (1,), torch.float32, dev, f"{name}(norm)")
    to = at
    if outs is not None:
        to, same, kept, where = _gradients(outs, name)
        if same != count or kept != kinds or where != dev:
            raise ValueError(f"{name}: outputs must be of the gradients' sizes and types, on their device")
    n = len(count)
    with _on(stream):
        ws, at_ws, size = _space(lib.kfac_grad_norm_workspace_size(n), norm.device, name)
    _call(lib.kfac_grad_clip(n, _pack_ptrs(at), _pack_ptrs(to), _pack_i64(count), _pack_kinds(kinds), max_norm, at_norm, at_ws,
                             size, _raw_stream(dev, stream)), name)
