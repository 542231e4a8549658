"""Layer bodies of a stack that are more than the stand-in.

LinearAttentionBody: v_l = W_out LinearAttention(q, k, v) with q, k, v one
projection of the aggregated row r_l, q and k normed per head and rotated by
position, a state of fixed size per layer, sequence and head.  Prompts run in
the chunked form over a ragged batch, decoding in the recurrent form with the
states in a pool of slots; both issue the same four kinds of launches and can
be captured in a CUDA graph with the stack around them.
"""
from __future__ import annotations

from contextlib import contextmanager, nullcontext
from dataclasses import dataclass
from typing import Sequence

import torch

from . import (
    ATTNRES_DEFAULT_EPS,
    attnres_linear,
    attnres_linear_attention,
    attnres_linear_attention_step,
    attnres_linear_attention_workspace_size,
    attnres_linear_workspace_size,
    attnres_qk_norm_rope,
)

__all__ = ["LinearAttentionWeights", "LinearAttentionBody"]


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


class LinearAttentionBody:
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
        if decode and cu_seqlens is not None:
            raise ValueError("cu_seqlens belong to prompts, slots to decoding")
        if not decode and slots is not None:
            raise ValueError("slots belong to decoding, cu_seqlens to prompts")
        if states.dim() != 5 or states.shape[0] != len(layers) or tuple(states.shape[2:]) != (heads, Dk, Dv):
            raise ValueError(f"states must be [{len(layers)}, n, {heads}, {Dk}, {Dv}]")
        w = layers[0].w_qkv
        dt, dev, d = w.dtype, w.device, w.shape[1]
        self.layers, self.states, self.log_decay = list(layers), states, log_decay
        self.heads, self.Dk, self.Dv, self.eps, self.scale, self.dev_err = heads, Dk, Dv, eps, scale, dev_err
        self.rope = dict(positions=positions, inv_freq=inv_freq, interleaved=interleaved)
        self.cu_seqlens, self.decode, self.slots = cu_seqlens, decode, slots
        width = heads * (2 * Dk + Dv)
        self.qkv = torch.empty((T, width), dtype=dt, device=dev)
        self.q = self.qkv[:, :heads * Dk].unflatten(1, (heads, Dk))
        self.k = self.qkv[:, heads * Dk:2 * heads * Dk].unflatten(1, (heads, Dk))
        self.v = self.qkv[:, 2 * heads * Dk:].unflatten(1, (heads, Dv))
        # the attention leaves rows outside every sequence or slot as they are:
        # zero, by each forward's first layer (issue)
        self.o = torch.zeros((T, heads, Dv), dtype=dt, device=dev)
        self._goes_on = None  # the layer that goes on from the last one issued
        n = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
        need = [n for l in self.layers for n in (attnres_linear_workspace_size(T, width, d, dt, w=l.w_qkv),
                                                 attnres_linear_workspace_size(T, d, heads * Dv, dt, w=l.w_out))]
        if not decode:
            need.append(attnres_linear_attention_workspace_size(T, heads, Dk, Dv, dt, n))
        # the four calls of a layer follow one another on one stream
        self.workspace = torch.empty(max(256, *need), dtype=torch.uint8, device=dev)

    def issue(self, layer: int, r: torch.Tensor, F: torch.Tensor, stream=None) -> None:
        w, state = self.layers[layer - 1], self.states[layer - 1]
        if layer != self._goes_on and (self.slots is not None or self.cu_seqlens is not None):
            # a forward (or a stage's part of one) begins: a row may have been
            # live in the last one and be padding now
            with _on(stream):
                self.o.zero_()
        self._goes_on = layer + 1
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
