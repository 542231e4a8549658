"""Layer bodies of a stack that are more than the stand-in.

LinearAttentionBody: v_l = W_out LinearAttention(q, k, v) with q, k, v one
projection of the aggregated row r_l, q and k normed per head and rotated by
position, a state of fixed size per layer, sequence and head.  Prompts run in
the chunked form over a ragged batch, decoding in the recurrent form with the
states in a pool of slots; both issue the same four kinds of launches and can
be captured in a CUDA graph with the stack around them.

GatedRecurrenceBody: v_l = W_out (h silu(g)) with x, f, g one projection of
the layer norm of r_l and h the gated linear recurrence of x by f, a state of
C channels per layer, sequence or slot; prompts and decoding as above.
"""
from __future__ import annotations

from contextlib import contextmanager, nullcontext
from dataclasses import dataclass
from typing import Sequence

import torch

from . import (
    ATTNRES_DEFAULT_EPS,
    attnres_gated_recurrence,
    attnres_gated_recurrence_step,
    attnres_layer_norm,
    attnres_linear,
    attnres_linear_attention,
    attnres_linear_attention_step,
    attnres_linear_attention_workspace_size,
    attnres_linear_workspace_size,
    attnres_qk_norm_rope,
)

__all__ = ["LinearAttentionWeights", "LinearAttentionBody", "GatedRecurrenceWeights", "GatedRecurrenceBody"]


@dataclass
class LinearAttentionWeights:
    """One layer: w_qkv [heads (2 Dk + Dv), d] (q, k and v side by side), w_out
    [d, heads Dv] of the stack's dtype; biases and gains float32 or None."""
    w_qkv: torch.Tensor
    w_out: torch.Tensor
    b_qkv: torch.Tensor | None = None
    b_out: torch.Tensor | None = None
    q_gain: torch.Tensor | None = None   # [Dk]
    k_gain: torch.Tensor | None = None


def _on(stream):
    """Makes torch's calls run on `stream` (None: the current one)."""
    if stream is None:
        return nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


class _Body:
    """What bodies with a state per sequence or slot share: T rows cut into
    sequences (prompts) or named by slots (decoding), and `o`, the mixer's
    output, whose rows outside all of them it leaves as they are."""

    def __init__(self, o: torch.Tensor, cu_seqlens: torch.Tensor | None, decode: bool, slots: torch.Tensor | None):
        if decode and cu_seqlens is not None:
            raise ValueError("cu_seqlens belong to prompts, slots to decoding")
        if not decode and slots is not None:
            raise ValueError("slots belong to decoding, cu_seqlens to prompts")
        self.o, self.cu_seqlens, self.decode, self.slots = o, cu_seqlens, decode, slots
        self._goes_on = None  # the layer that goes on from the last one issued

    def _begin(self, layer: int, stream) -> None:
        if layer != self._goes_on and (self.slots is not None or self.cu_seqlens is not None):
            # a forward (or a stage's part of one) begins: a row may have been
            # live in the last one and be padding now
            with _on(stream):
                self.o.zero_()
        self._goes_on = layer + 1

    @contextmanager
    def idle(self):
        """Within it no row is of any sequence or slot: forwards issue the same
        kernels and change no state (StackForward.capture's eager run)."""
        kept = self.slots, self.cu_seqlens
        if self.decode:
            self.slots = torch.full((self.o.shape[0],), -1, dtype=torch.int32, device=self.o.device)
        else:
            n = 1 if self.cu_seqlens is None else self.cu_seqlens.numel() - 1
            self.cu_seqlens = torch.zeros(n + 1, dtype=torch.int32, device=self.o.device)
        try:
            yield
        finally:
            self.slots, self.cu_seqlens = kept


class LinearAttentionBody(_Body):
    """The body of every layer of one stack over T rows.

    layers: the L layers' weights; log_decay [heads] float32; states: [L,
    n, heads, Dk, Dv] float32, of the n sequences (prompts) or slots
    (decoding), read and updated in place by every forward (a first prompt
    starts from zeros); positions [T] int64 and inv_freq [rot / 2] float32, or
    both None (no rotation): a caller may overwrite positions between
    forwards, captured or not.

    Prompts: cu_seqlens [n + 1] int32 on the device cuts the T rows into
    sequences (None: one).  Decoding (decode=True): row b is the next token of
    the sequence in slot slots[b] ([T] int32; None: slot b).  Rows outside
    every sequence or slot give v = b_out.  A caller may overwrite both between
    forwards, captured or not (not between the layers of one).

    The body's buffers and workspace belong to one forward at a time: two
    stacks, or two captured graphs of one, that run at once need a body each.
    """

    def __init__(self, layers: Sequence[LinearAttentionWeights], T: int, heads: int, Dk: int, Dv: int,
                 log_decay: torch.Tensor, states: torch.Tensor, positions: torch.Tensor | None = None,
                 inv_freq: torch.Tensor | None = None, interleaved: bool = False,
                 cu_seqlens: torch.Tensor | None = None, decode: bool = False, slots: torch.Tensor | None = None,
                 eps: float = ATTNRES_DEFAULT_EPS, scale: float | None = None, dev_err: torch.Tensor | None = None):
        if states.dim() != 5 or states.shape[0] != len(layers) or tuple(states.shape[2:]) != (heads, Dk, Dv):
            raise ValueError(f"states must be [{len(layers)}, n, {heads}, {Dk}, {Dv}]")
        w = layers[0].w_qkv
        dt, dev, d = w.dtype, w.device, w.shape[1]
        self.layers, self.states, self.log_decay = list(layers), states, log_decay
        self.heads, self.Dk, self.Dv, self.eps, self.scale, self.dev_err = heads, Dk, Dv, eps, scale, dev_err
        self.rope = dict(positions=positions, inv_freq=inv_freq, interleaved=interleaved)
        width = heads * (2 * Dk + Dv)
        self.qkv = torch.empty((T, width), dtype=dt, device=dev)
        self.q = self.qkv[:, :heads * Dk].unflatten(1, (heads, Dk))
        self.k = self.qkv[:, heads * Dk:2 * heads * Dk].unflatten(1, (heads, Dk))
        self.v = self.qkv[:, 2 * heads * Dk:].unflatten(1, (heads, Dv))
        # the attention leaves rows outside every sequence or slot as they are:
        # zero, by each forward's first layer (_begin)
        super().__init__(torch.zeros((T, heads, Dv), dtype=dt, device=dev), cu_seqlens, decode, slots)
        n = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        need = [n for l in self.layers for n in (attnres_linear_workspace_size(T, width, d, dt, w=l.w_qkv),
                                                 attnres_linear_workspace_size(T, d, heads * Dv, dt, w=l.w_out))]
        if not decode:
            need.append(attnres_linear_attention_workspace_size(T, heads, Dk, Dv, dt, n))
        # the four calls of a layer follow one another on one stream
        self.workspace = torch.empty(max(256, *need), dtype=torch.uint8, device=dev)

    def issue(self, layer: int, r: torch.Tensor, F: torch.Tensor, stream=None) -> None:
        w, state = self.layers[layer - 1], self.states[layer - 1]
        self._begin(layer, stream)
        attnres_linear(r, w.w_qkv, self.qkv, bias=w.b_qkv, workspace=self.workspace, dev_err=self.dev_err, stream=stream)
        attnres_qk_norm_rope(self.q, self.k, self.q, self.k, q_gain=w.q_gain, k_gain=w.k_gain, eps=self.eps,
                             stream=stream, **self.rope)
        if self.decode:
            attnres_linear_attention_step(self.q, self.k, self.v, self.log_decay, state, self.o, slots=self.slots,
                                          scale=self.scale, stream=stream)
        else:
            attnres_linear_attention(self.q, self.k, self.v, self.log_decay, self.o, cu_seqlens=self.cu_seqlens,
                                     initial_state=state, final_state=state, scale=self.scale,
                                     workspace=self.workspace, dev_err=self.dev_err, stream=stream)
        attnres_linear(self.o.flatten(1), w.w_out, F, bias=w.b_out, workspace=self.workspace, dev_err=self.dev_err,
                       stream=stream)


@dataclass
class GatedRecurrenceWeights:
    """One layer: w_in [3 C, d] (x, forget gate and output gate side by side),
    w_out [d, C] of the stack's dtype; biases, gain and bias of the norm
    float32 or None."""
    w_in: torch.Tensor
    w_out: torch.Tensor
    b_in: torch.Tensor | None = None
    b_out: torch.Tensor | None = None
    norm_gain: torch.Tensor | None = None   # [d]
    norm_bias: torch.Tensor | None = None   # [d]


class GatedRecurrenceBody(_Body):
    """The body of every layer of one stack over T rows.

    layers: the L layers' weights; states: [L, n, C] float32, of the n
    sequences (prompts) or slots (decoding), read and updated in place by every
    forward (a first prompt starts from zeros).  cu_seqlens, decode and slots,
    rows outside every sequence or slot (v = b_out), and what a caller may
    overwrite between forwards: as for LinearAttentionBody.

    The body's buffers and workspace belong to one forward at a time: two
    stacks, or two captured graphs of one, that run at once need a body each.
    """

    def __init__(self, layers: Sequence[GatedRecurrenceWeights], T: int, states: torch.Tensor,
                 cu_seqlens: torch.Tensor | None = None, decode: bool = False, slots: torch.Tensor | None = None,
                 eps: float = ATTNRES_DEFAULT_EPS, dev_err: torch.Tensor | None = None):
        w = layers[0].w_in
        dt, dev, d, C = w.dtype, w.device, w.shape[1], w.shape[0] // 3
        if states.dim() != 3 or states.shape[0] != len(layers) or states.shape[2] != C:
            raise ValueError(f"states must be [{len(layers)}, n, {C}]")
        super().__init__(torch.zeros((T, C), dtype=dt, device=dev), cu_seqlens, decode, slots)
        self.layers, self.states, self.eps, self.dev_err = list(layers), states, eps, dev_err
        self.normed = torch.empty((T, d), dtype=dt, device=dev)
        self.xfg = torch.empty((T, 3 * C), dtype=dt, device=dev)
        self.x, self.forget, self.gate = self.xfg.split(C, 1)
        need = [n for l in self.layers for n in (attnres_linear_workspace_size(T, 3 * C, d, dt, w=l.w_in),
                                                 attnres_linear_workspace_size(T, d, C, dt, w=l.w_out))]
        # the four calls of a layer follow one another on one stream
        self.workspace = torch.empty(max(256, *need), dtype=torch.uint8, device=dev)

    def issue(self, layer: int, r: torch.Tensor, F: torch.Tensor, stream=None) -> None:
        w, state = self.layers[layer - 1], self.states[layer - 1]
        self._begin(layer, stream)
        attnres_layer_norm(r, self.normed, gain=w.norm_gain, bias=w.norm_bias, eps=self.eps, stream=stream)
        attnres_linear(self.normed, w.w_in, self.xfg, bias=w.b_in, workspace=self.workspace, dev_err=self.dev_err,
                       stream=stream)
        if self.decode:
            attnres_gated_recurrence_step(self.x, self.forget, state, self.o, gate=self.gate, slots=self.slots,
                                          stream=stream)
        else:
            attnres_gated_recurrence(self.x, self.forget, self.o, gate=self.gate, cu_seqlens=self.cu_seqlens,
                                     initial_state=state, final_state=state, dev_err=self.dev_err, stream=stream)
        attnres_linear(self.o, w.w_out, F, bias=w.b_out, workspace=self.workspace, dev_err=self.dev_err, stream=stream)
