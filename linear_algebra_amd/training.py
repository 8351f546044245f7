"""Training an encoder layer under the preconditioner: attention as a
differentiable function, a linear layer that keeps its input in 8 bits, layer
norm, the gated feed-forward projections, and the clipping of the gradients to
a norm.

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
               kfac_checkpoint_store, kfac_gated_backward, kfac_gated_forward, kfac_grad_clip, kfac_layer_norm_backward,
               kfac_layer_norm_forward)


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


def _differentiable(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _matrix(t, d):
    """t as a matrix of rows of d elements, each row contiguous and apart from the others (a view where that can be)."""
    t = t.reshape(-1, d)
    return t if t.stride(1) == 1 and t.stride(0) >= d else t.contiguous()


# (A call goes through its autograd function where nothing asks for a gradient
# too: what a kernel writes is known to torch's forward mode and tracing as that
# function's output alone.  `keep`: whether a backward pass may follow.)

class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, d, keep):
        rows = _matrix(x, d)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if not keep:
            kfac_layer_norm_forward(rows, y.view(rows.shape), weight=weight, bias=bias, eps=eps)
            return y
        mean, rstd = (torch.empty(rows.shape[0], dtype=torch.float32, device=x.device) for _ in range(2))
        kfac_layer_norm_forward(rows, y.view(rows.shape), mean, rstd, weight=weight, bias=bias, eps=eps)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.d = d
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        rows = _matrix(x.detach(), ctx.d)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if ctx.needs_input_grad[0] else None
        dw = torch.empty_like(weight) if ctx.needs_input_grad[1] else None
        db = torch.empty_like(bias) if ctx.needs_input_grad[2] else None
        kfac_layer_norm_backward(_matrix(dy.detach(), ctx.d), rows, mean, rstd, None if dx is None else dx.view(rows.shape),
                                 weight=weight, dweight=dw, dbias=db)
        return *_final((dx, dw, db), [t for t in (dy, x, weight) if t is not None]), None, None, None


def layer_norm(x, weight=None, bias=None, eps=1e-5, dims=1):
    """Layer norm over the last `dims` dimensions of x (float32 or bfloat16),
    differentiable once in x, weight and bias, which have those dimensions and
    are float32 or of x's type, both alike.  Tangents (forward mode) and
    functional transforms raise."""
    d = 1
    for n in x.shape[x.dim() - dims:]:
        d *= int(n)   # (a tensor while a program is traced)
    if x.dim() < dims or any(t is not None and t.shape != x.shape[x.dim() - dims:] for t in (weight, bias)):
        raise ValueError("layer_norm: weight and bias must have the shape of x's last dimensions")
    weight, bias = (None if t is None else t.contiguous().view(-1) for t in (weight, bias))
    return _LayerNorm.apply(x, weight, bias, eps, d, _differentiable(x, weight, bias))


class LayerNorm(torch.nn.LayerNorm):
    """torch.nn.LayerNorm on the library's kernels (see :func:`layer_norm`)."""

    def forward(self, x):
        if x.shape[x.dim() - len(self.normalized_shape):] != self.normalized_shape:
            raise ValueError(f"LayerNorm: expected the last dimensions {tuple(self.normalized_shape)}")
        return layer_norm(x, self.weight, self.bias, self.eps, len(self.normalized_shape))


def _words(t):
    """t contiguous, beginning on 4 bytes."""
    t = t.contiguous()
    return t if t.data_ptr() % 4 == 0 else t.clone()


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, activation, unrounded, module, keep):
        rows = _words(x.reshape(-1, weight.shape[1]))
        wide = rows.shape[0], weight.shape[0]
        w = _words(weight.to(x.dtype))
        h = torch.empty(*x.shape[:-1], wide[1] // 2, dtype=x.dtype, device=x.device)
        pre = torch.empty(wide, dtype=x.dtype, device=x.device) if keep else None
        kfac_gated_forward(rows, w, h.view(wide[0], wide[1] // 2), bias=None if bias is None else bias.float().contiguous(),
                           pre=pre, activation=activation)
        if not keep:
            return h
        ctx.save_for_backward(x, weight, bias, pre)
        ctx.activation, ctx.unrounded, ctx.module = activation, unrounded, module
        return h

    @staticmethod
    def backward(ctx, dh):
        x, weight, bias, pre = ctx.saved_tensors
        rows = _words(x.detach().reshape(-1, weight.shape[1]))
        w = _words(weight.detach().to(x.dtype))
        dpre = torch.empty_like(pre, dtype=torch.float32 if ctx.unrounded else None)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if ctx.needs_input_grad[0] else None
        # the weight's gradient in its own type, with no rounding to the rows' type before
        kind = weight.dtype if weight.dtype in (torch.float32, x.dtype) else torch.float32
        dw = torch.empty(weight.shape, dtype=kind, device=x.device) if ctx.needs_input_grad[1] else None
        db = torch.empty(bias.shape, dtype=torch.float32, device=x.device) if ctx.needs_input_grad[2] else None
        kfac_gated_backward(dh.detach().reshape(pre.shape[0], weight.shape[0] // 2).contiguous(), rows, w, pre, dpre,
                            None if dx is None else dx.view(rows.shape), dw, db, activation=ctx.activation)
        if ctx.module is not None:
            for hook in ctx.module.output_grad_hooks:
                hook(ctx.module, dpre.to(x.dtype))
        dw = None if dw is None else dw.to(weight.dtype)
        db = None if db is None else db.to(bias.dtype)
        return *_final((dx, dw, db), [t for t in (dh, x, weight, bias) if t is not None]), None, None, None, None


def gated_linear(x, weight, bias=None, activation="silu", unrounded=False):
    """act(g) u with [g | u] = x weight^T + bias over the last dimension of x
    (float32 or bfloat16), weight [2 width, d] with the gate's rows first;
    differentiable once in x, weight and bias.  Tangents (forward mode) and
    functional transforms raise.  Weight and bias may be float32 while x is
    bfloat16.  activation: silu, gelu, gelu_tanh, relu or sigmoid.
    unrounded: whether the gradient of [g | u] enters the gradients of a
    bfloat16 x and of the weight in float32 instead of in bfloat16 (three times
    the work of these products)."""
    return _gated(x, weight, bias, activation, unrounded, None)


def _gated(x, weight, bias, activation, unrounded, module):
    if weight.dim() != 2 or weight.shape[0] % 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("gated_linear: expected x [..., d] and weight [2 width, d]")
    return _Gated.apply(x, weight, bias, activation, unrounded, module, _differentiable(x, weight, bias))


class GatedLinear(torch.nn.Linear):
    """The two projections of a gated feed-forward block as one layer: weight
    [2 width, d], the gate's rows first, and the output act(g) u of width
    `width` (see :func:`gated_linear`).  Under
    :class:`linear_algebra_amd.kfac_preconditioner.KFACPreconditioner` it is a
    linear layer whose output is [g | u]: its factor G is that of [g | u]'s
    gradient, which the backward pass hands to each of `output_grad_hooks` (as
    hook(module, gradient [rows, 2 width] in the input's type))."""

    unrounded = False   # (of layers stored before there was a choice)

    def __init__(self, in_features, width, bias=True, activation="silu", device=None, dtype=None, unrounded=False):
        super().__init__(in_features, 2 * width, bias=bias, device=device, dtype=dtype)
        self.width, self.activation, self.unrounded = width, activation, unrounded
        self.output_grad_hooks = []

    def forward(self, x):
        return _gated(x, self.weight, self.bias, self.activation, self.unrounded, self)

    def extra_repr(self):
        return f"in_features={self.in_features}, width={self.width}, bias={self.bias is not None}, activation={self.activation}"


def clip_grad_norm_(parameters, max_norm):
    """Scales the gradients of the parameters in place so that their norm,
    taken together, is at most max_norm; returns the norm that they had, a
    tensor that nothing has waited for.  At most 4096 gradients, float32 or
    bfloat16, on one GPU, of separate memory (a parameter given twice is
    refused)."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    if not grads:
        return torch.tensor(0.0)
    with torch.no_grad():
        flat, copies = [], []
        for g in grads:
            if not g.is_contiguous():
                # the same elements in the order in which they lie in memory
                v = g.detach().permute(sorted(range(g.dim()), key=lambda k: -g.stride(k)))
                if not v.is_contiguous():
                    v = g.detach().contiguous()
                    copies.append((g, v))
                g = v
            flat.append(g)
        norm = torch.empty(1, dtype=torch.float32, device=grads[0].device)
        kfac_grad_clip(flat, float(max_norm), norm)
        for g, v in copies:
            g.copy_(v)
        # the kernels wrote them behind autograd's back
        torch.autograd.graph.increment_version(grads)
    return norm.reshape(())
