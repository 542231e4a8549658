"""One layer of depth-wise attention, and the operators of a layer body, as
differentiable torch operations.

`aggregate(H, w)` returns r = sum_s softmax_s(w . RMSNorm(H_s)) H_s for a
[S, T, d] stack of sources (float32 or bfloat16) and an fp32 pseudo-query
[d], and takes part in torch autograd: the forward runs attnres_aggregate,
the backward attnres_aggregate_backward (the forward recomputed inside it,
as under activation checkpointing: only H and w are kept).  Both run in the
library's kernels; torch only allocates the outputs and the backward's
workspace.  Gradients: dH in the sources' dtype, dw in fp32 (summed over
tokens in a fixed order, so bit-reproducible).  The incoming gradient of r
is taken in the sources' dtype (the backward kernel reads it so): an fp32
gradient for bf16 sources is rounded to bf16 first.

`linear`, `qk_norm_rope`, `linear_attention`, `layer_norm` and
`gated_recurrence` wrap the calls of the same names the same way: nothing but
the inputs is kept (of the recurrence also its states ahead of every 64th
row), the backward recomputes what it needs, incoming gradients are taken in
the tensors' dtype, and gradients nobody asks for are not formed.  They can be differentiated once.
Before a backward is captured in a CUDA graph, let go of eager graphs of the
same leaves (torch runs their accumulation on the stream they were made on).

`clip_grad_norm` ends a training step: it clips the gradients that leaves hold.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (
    ATTNRES_DEFAULT_EPS,
    ATTNRES_RECURRENCE_CHUNK,
    attnres_aggregate,
    attnres_aggregate_backward,
    attnres_gated_recurrence,
    attnres_gated_recurrence_backward,
    attnres_grad_clip,
    attnres_layer_norm,
    attnres_layer_norm_backward,
    attnres_linear,
    attnres_linear_attention,
    attnres_linear_attention_backward,
    attnres_linear_backward,
    attnres_qk_norm_rope,
    attnres_qk_norm_rope_backward,
)

__all__ = ["AttnResAggregate", "aggregate", "linear", "qk_norm_rope", "linear_attention", "layer_norm",
           "gated_recurrence", "clip_grad_norm"]


class AttnResAggregate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H: torch.Tensor, w: torch.Tensor, eps: float) -> torch.Tensor:
        if H.dim() != 3:
            raise ValueError("H must be [S, T, d]")
        H = H.contiguous()
        S, T, d = H.shape
        r = torch.empty((T, d), dtype=H.dtype, device=H.device)
        attnres_aggregate(H, w, r, None, eps=eps)
        ctx.save_for_backward(H, w)
        ctx.eps = eps
        return r

    @staticmethod
    def backward(ctx, grad_r: torch.Tensor):
        H, w = ctx.saved_tensors
        grad_r = grad_r.to(H.dtype).contiguous()
        grad_H = torch.empty_like(H)
        grad_w = torch.empty_like(w)
        attnres_aggregate_backward(H, w, grad_r, grad_H, grad_w, eps=ctx.eps)
        return (grad_H if ctx.needs_input_grad[0] else None,
                grad_w if ctx.needs_input_grad[1] else None, None)


def aggregate(H: torch.Tensor, w: torch.Tensor, eps: float = ATTNRES_DEFAULT_EPS) -> torch.Tensor:
    """r = sum_s softmax_s(w . RMSNorm(H_s)) H_s, differentiable in H and w."""
    return AttnResAggregate.apply(H, w, eps)


def _rows_contiguous(t: torch.Tensor) -> torch.Tensor:
    """t itself where the calls take it (rows contiguous behind the first
    dimension, in order), or a contiguous copy."""
    inner = 1
    for n, s in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n > 1 and s != inner:
            return t.contiguous()
        inner *= n
    return t if t.shape[0] <= 1 or t.stride(0) >= inner else t.contiguous()


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, activation):
        x, w = _rows_contiguous(x), w.contiguous()
        out = torch.empty((x.shape[0], w.shape[0]), dtype=x.dtype, device=x.device)
        attnres_linear(x, w, out, bias=bias, residual=None if residual is None else _rows_contiguous(residual),
                       activation=activation)
        ctx.save_for_backward(x, w, bias)
        ctx.activation = activation
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, w, bias = ctx.saved_tensors
        need_x, need_w, need_b, need_r, _ = ctx.needs_input_grad
        grad = _rows_contiguous(grad.to(x.dtype))
        gx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_x else None
        gw = torch.empty_like(w) if need_w else None
        gb = torch.empty_like(bias) if need_b else None
        attnres_linear_backward(x, w, grad, gx, gw, gb, bias=bias, activation=ctx.activation)
        return gx, gw, gb, grad if need_r else None, None


def linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None,
           residual: torch.Tensor | None = None, activation: str = "none") -> torch.Tensor:
    """activation(x w^T + bias) + residual over x's last dimension; w [N, K]
    of x's dtype, bias [N] float32, residual of the result's shape."""
    lead = x.shape[:-1]
    flat = None if residual is None else residual.reshape(-1, w.shape[0])
    return _Linear.apply(x.reshape(-1, x.shape[-1]), w, bias, flat, activation).reshape(*lead, w.shape[0])


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_gain, k_gain, positions, inv_freq, interleaved, eps):
        q, k = _rows_contiguous(q), _rows_contiguous(k)
        outs = [torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k)]
        if ctx.needs_input_grad[5]:
            raise ValueError("inv_freq is a constant: it gets no gradient")
        ctx.rope = dict(interleaved=interleaved, eps=eps)
        attnres_qk_norm_rope(q, k, *outs, q_gain=q_gain, k_gain=k_gain, positions=positions, inv_freq=inv_freq, **ctx.rope)
        # (saved, so that torch refuses a backward whose angles were written over)
        ctx.save_for_backward(q, k, q_gain, k_gain, positions, inv_freq)
        return tuple(outs)

    @staticmethod
    @once_differentiable
    def backward(ctx, gq, gk):
        q, k, q_gain, k_gain, positions, inv_freq = ctx.saved_tensors
        need_q, need_k, need_qg, need_kg = ctx.needs_input_grad[:4]
        # (a gain's gradient comes with its tensor's)
        q, k = q if need_q or need_qg else None, k if need_k or need_kg else None
        grads = [None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k)]
        gains = [torch.empty_like(g) if need else None for g, need in ((q_gain, need_qg), (k_gain, need_kg))]
        gq, gk = (None if t is None else _rows_contiguous(g.to(t.dtype)) for g, t in ((gq, q), (gk, k)))
        attnres_qk_norm_rope_backward(q, k, gq, gk, *grads,
                                      q_gain=q_gain, k_gain=k_gain, grad_q_gain=gains[0], grad_k_gain=gains[1],
                                      positions=positions, inv_freq=inv_freq, **ctx.rope)
        return (*grads, *gains, None, None, None, None)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_gain: torch.Tensor | None = None,
                 k_gain: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                 inv_freq: torch.Tensor | None = None, interleaved: bool = False,
                 eps: float = ATTNRES_DEFAULT_EPS) -> tuple[torch.Tensor, torch.Tensor]:
    """RMSNorm of q's and k's heads [T, heads, D] and their rotation, differentiable in q, k and the gains."""
    return _QkNormRope.apply(q, k, q_gain, k_gain, positions, inv_freq, interleaved, eps)


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, cu_seqlens, initial_state, scale):
        q, k, v = _rows_contiguous(q), _rows_contiguous(k), _rows_contiguous(v)
        n = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        if cu_seqlens is not None:
            out.zero_()  # rows outside every sequence
        final = torch.empty((n, q.shape[1], q.shape[2], v.shape[2]), dtype=torch.float32, device=q.device)
        initial_state = None if initial_state is None else initial_state.contiguous()
        attnres_linear_attention(q, k, v, log_decay, out, cu_seqlens=cu_seqlens, initial_state=initial_state,
                                 final_state=final, scale=scale)
        ctx.save_for_backward(q, k, v, log_decay, cu_seqlens, initial_state)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_final):
        q, k, v, log_decay, cu_seqlens, initial_state = ctx.saved_tensors
        if grad_out is None:
            grad_out = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
        make = torch.empty if cu_seqlens is None else torch.zeros
        need_q, need_k, need_v, _, _, need_0, _ = ctx.needs_input_grad
        # (the initial state's gradient comes with v's)
        grads = [make(t.shape, dtype=t.dtype, device=t.device) if need else None
                 for t, need in ((q, need_q), (k, need_k), (v, need_v or need_0))]
        g0 = torch.empty_like(initial_state) if need_0 else None
        attnres_linear_attention_backward(q, k, v, log_decay, _rows_contiguous(grad_out.to(v.dtype)), *grads,
                                          cu_seqlens=cu_seqlens, initial_state=initial_state,
                                          grad_final_state=None if grad_final is None else grad_final.contiguous(),
                                          grad_initial_state=g0, scale=ctx.scale)
        return (*grads, None, None, g0, None)


def linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                     cu_seqlens: torch.Tensor | None = None, initial_state: torch.Tensor | None = None,
                     scale: float | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(out [T, H, Dv], final states [num_seqs, H, Dk, Dv] float32) of
    attnres_linear_attention, differentiable in q, k, v and the initial
    states; rows outside every sequence are zero and get zero gradients."""
    return _LinearAttention.apply(q, k, v, log_decay, cu_seqlens, initial_state, scale)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gain, bias, eps):
        x = _rows_contiguous(x)
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        attnres_layer_norm(x, out, gain=gain, bias=bias, eps=eps)
        ctx.save_for_backward(x, gain)
        ctx.eps = eps
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        x, gain = ctx.saved_tensors
        need_x, need_g, need_b, _ = ctx.needs_input_grad
        gx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_x else None
        gg, gb = (torch.empty(x.shape[1], dtype=torch.float32, device=x.device) if need else None for need in (need_g, need_b))
        attnres_layer_norm_backward(x, _rows_contiguous(grad.to(x.dtype)), gx, gain=gain, grad_gain=gg, grad_bias=gb,
                                    eps=ctx.eps)
        return gx, gg, gb, None


def layer_norm(x: torch.Tensor, gain: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = ATTNRES_DEFAULT_EPS) -> torch.Tensor:
    """gain (x - mean) / sqrt(var + eps) + bias over x's last dimension; gain and bias [d] float32 or None."""
    return _LayerNorm.apply(x.reshape(-1, x.shape[-1]), gain, bias, eps).reshape(x.shape)


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, forget, gate, cu_seqlens, initial_state):
        x, forget = _rows_contiguous(x), _rows_contiguous(forget)
        gate = None if gate is None else _rows_contiguous(gate)
        n = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        T, C = x.shape
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if cu_seqlens is not None:
            out.zero_()  # rows outside every sequence
        final = torch.empty((n, C), dtype=torch.float32, device=x.device)
        chunk = None
        if any(ctx.needs_input_grad):
            chunk = torch.empty((-(-T // ATTNRES_RECURRENCE_CHUNK), C), dtype=torch.float32, device=x.device)
        initial_state = None if initial_state is None else initial_state.contiguous()
        attnres_gated_recurrence(x, forget, out, gate=gate, cu_seqlens=cu_seqlens, initial_state=initial_state,
                                 final_state=final, chunk_states=chunk)
        ctx.save_for_backward(x, forget, gate, cu_seqlens, initial_state, chunk)
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_final):
        x, forget, gate, cu_seqlens, initial_state, chunk = ctx.saved_tensors
        if grad_out is None:
            grad_out = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        make = torch.empty if cu_seqlens is None else torch.zeros
        need_x, need_f, need_g, _, need_0 = ctx.needs_input_grad
        grads = [make(x.shape, dtype=x.dtype, device=x.device) if need else None for need in (need_x, need_f, need_g)]
        g0 = torch.empty_like(initial_state) if need_0 else None
        attnres_gated_recurrence_backward(x, forget, chunk, _rows_contiguous(grad_out.to(x.dtype)), *grads, gate=gate,
                                          cu_seqlens=cu_seqlens, initial_state=initial_state,
                                          grad_final_state=None if grad_final is None else grad_final.contiguous(),
                                          grad_initial_state=g0)
        return (*grads, None, g0)


def gated_recurrence(x: torch.Tensor, forget: torch.Tensor, gate: torch.Tensor | None = None,
                     cu_seqlens: torch.Tensor | None = None,
                     initial_state: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(out [T, C], final states [num_seqs, C] float32) of
    attnres_gated_recurrence, differentiable in x, forget, gate and the
    initial states; rows outside every sequence are zero and get zero
    gradients."""
    return _GatedRecurrence.apply(x, forget, gate, cu_seqlens, initial_state)


def clip_grad_norm(leaves, max_norm: float) -> torch.Tensor:
    """The 2-norm [1] float32 of all the gradients that `leaves` hold, which are
    then clipped in place to max_norm (attnres_grad_clip).  Nothing is copied to
    the host.  A gradient that is not contiguous is replaced by a contiguous
    copy first.

    Not as in torch.nn.utils.clip_grad_norm_: the factor is max_norm / norm
    without an addend, a norm that is not finite leaves the gradients as they
    are, and leaves without any gradient are a ValueError."""
    leaves = [leaves] if isinstance(leaves, torch.Tensor) else list(leaves)
    grads = []
    for p in {id(p): p for p in leaves}.values():  # a leaf named twice counts once
        if p.grad is not None:
            if not p.grad.is_contiguous():
                p.grad = p.grad.contiguous()
            grads.append(p.grad)
    if not grads:
        raise ValueError("none of the leaves holds a gradient")
    norm = torch.empty(1, dtype=torch.float32, device=grads[0].device)
    attnres_grad_clip(grads, max_norm, norm)
    return norm
