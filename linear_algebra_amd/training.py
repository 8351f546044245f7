"""Training an encoder layer under the preconditioner: attention as a
differentiable function, and a linear layer that keeps its input in 8 bits.

Between the forward and the backward pass attention keeps its output and one
logarithm per query (the probabilities are formed again), and
:class:`CheckpointLinear` keeps 33/32 bytes per input element; the kept input
serves the weight gradient and, under
:class:`linear_algebra_amd.kfac_preconditioner.KFACPreconditioner`, the
factor A of the layer.
"""
from __future__ import annotations

import torch

from . import (kfac_attention_backward, kfac_attention_forward, kfac_checkpoint_empty, kfac_checkpoint_grad,
               kfac_checkpoint_store)


def _rows16(t):
    """The tensor itself where its last dimension is contiguous, every row
    starts on 16 bytes and rows lie within the kernels' largest stride (2^30 /
    128 bytes), else a contiguous copy."""
    size = t.element_size()
    if t.stride(3) == 1 and t.data_ptr() % 16 == 0 and all(t.stride(n) * size % 16 == 0 for n in range(3)) \
            and t.stride(1) * size <= 1 << 23:
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _Final(torch.autograd.Function):
    """The first n tensors as functions of the others, which cannot be differentiated."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.detach() for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("linear_algebra_amd.training: second derivatives are not formed")


def _final(grads, sources):
    """The gradients of a kernel's call.  In a pass that builds a graph of its
    own (create_graph), differentiating them raises, on every way to what the
    sources depend on, instead of taking them for constants."""
    if not torch.is_grad_enabled():
        return grads
    some = [g for g in grads if g is not None]
    linked = iter(_Final.apply(len(some), *some, *sources))
    return tuple(None if g is None else next(linked) for g in grads)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, bias, lens, form):
        q, k, v = (_rows16(t) for t in (q, k, v))
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[0], q.shape[2], q.shape[1], dtype=torch.float32, device=q.device)
        kfac_attention_forward(q, k, v, out, lse, bias=bias, lens=lens, **form)
        ctx.save_for_backward(q, k, v, out, lse, bias, lens)
        ctx.form = form
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse, bias, lens = ctx.saved_tensors
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        dbias = None if bias is None else torch.empty_like(bias)
        kfac_attention_backward(q, k, v, out, lse, _rows16(dout), dq, dk, dv, dbias, bias=bias, lens=lens,
                                **ctx.form)
        return *_final((dq, dk, dv, dbias), (dout, out)), None, None


def attention(q, k, v, scale=None, causal=False, lens=None, bias=None, borders=None, two_sided=True):
    """Softmax attention of q [batch, len_q, heads, dim] over k, v [batch,
    len_k, kv_heads, dim], differentiable once in q, k, v and the bias table
    (arguments as in kfac_attention_forward)."""
    if borders is not None:
        # (a copy: the backward pass reads them too)
        borders = tuple(borders.tolist() if hasattr(borders, "tolist") else borders)
    form = dict(scale=scale, causal=causal, borders=borders, two_sided=two_sided)
    return _Attention.apply(q, k, v, None if bias is None else bias.contiguous(), lens, form)


class _KeptLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, module):
        rows = x.reshape(-1, x.shape[-1]).contiguous()
        codes, scales = kfac_checkpoint_empty(rows.shape[0], rows.shape[1] + (bias is not None), x.device)
        if rows.shape[0]:
            kfac_checkpoint_store([rows], [codes], [scales], ones=bias is not None)
        module.kept = (codes, scales, rows.shape[0], x.shape[0])
        y = torch.nn.functional.linear(x, weight.to(x.dtype), None if bias is None else bias.to(x.dtype))
        # an output that stands for the others in _final without keeping them
        empty = y.new_empty(0)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(weight, codes, scales, empty)
        ctx.has_bias = bias is not None
        return y, empty

    @staticmethod
    def backward(ctx, gy, _):
        weight, codes, scales, empty = ctx.saved_tensors
        dx = torch.matmul(gy, weight.to(gy.dtype)) if ctx.needs_input_grad[0] else None
        if not (ctx.needs_input_grad[1] or ctx.needs_input_grad[2]):
            return dx, None, None, None
        rows = gy.reshape(-1, gy.shape[-1]).contiguous()
        if rows.shape[0]:
            mat = torch.empty(weight.shape[0], codes.shape[1], dtype=torch.float32, device=gy.device)
            kfac_checkpoint_grad([rows], [codes], [scales], [mat])
        else:
            mat = torch.zeros(weight.shape[0], codes.shape[1], dtype=torch.float32, device=gy.device)
        dw = mat[:, :weight.shape[1]].to(weight.dtype).contiguous()
        db = mat[:, -1].to(weight.dtype).contiguous() if ctx.has_bias else None
        return dx, *_final((dw, db), (gy, empty)), None


class CheckpointLinear(torch.nn.Linear):
    """A linear layer whose input is kept in 8 bits for the backward pass.
    The output is that of ``torch.nn.Linear``; the weight and bias gradients
    (formed in one product, the bias as the gradient of a column of ones) and
    the preconditioner's factor A are those of the kept input.  The weights
    may be float32 while the input is bfloat16.  The input's gradient can be
    differentiated again, the weight and bias gradients cannot.  ``kept`` holds
    the last training pass's checkpoint: codes, scales, rows, batch."""

    kept = None

    def forward(self, x):
        if not (self.training and torch.is_grad_enabled()):
            return torch.nn.functional.linear(x, self.weight.to(x.dtype),
                                              None if self.bias is None else self.bias.to(x.dtype))
        return _KeptLinear.apply(x, self.weight, self.bias, self)[0]
