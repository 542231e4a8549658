"""Block Attention Residuals (Block AttnRes) depth aggregation for GB300.

A thin Python binding of ``libattnres`` (C ABI in ``include/attnres.h``);
the functions keep the C names.  torch supplies device memory and streams
only: tensors are passed as device pointers, the current torch CUDA stream
is used unless one is given, and every step of the computation runs in the
library's sm_103a kernels.  Importing raises if the library is missing.

What is computed ("Kimi K3 deep-dive series (2): AttnRes and Stable
LatentMoE", §2; Kimi K3 chaptered tutorial, ch. 4.3 Eq. 10):
    a_l = softmax_s(w_l . RMSNorm(h_s)),  r_l = sum_s a_l[s] h_s
over the sources [h_0, b_1 .. b_{n-1}, partial sum of the current block].
"""
from __future__ import annotations

import ctypes
from typing import Sequence

import torch

from . import _native as _N
from ._native import (  # noqa: F401
    ATTNRES_ACT_GELU,
    ATTNRES_ACT_GELU_TANH,
    ATTNRES_ACT_NONE,
    ATTNRES_ACT_SILU,
    ATTNRES_BF16,
    ATTNRES_DEFAULT_EPS,
    ATTNRES_DEVERR_WAIT_TIMEOUT,
    ATTNRES_F32,
    ATTNRES_MAX_BLOCKS,
    ATTNRES_MAX_SOURCES,
    ATTNRES_STATE_EARLY_LOADS,
    AttnresError,
    LIB_PATH,
)

__all__ = [
    "attnres_aggregate", "attnres_aggregate_backward", "attnres_aggregate_backward_workspace_size",
    "attnres_interblock", "attnres_interblock_workspace_size", "attnres_intrablock_step", "attnres_num_sources", "attnres_layer_sources", "attnres_block_step",
    "attnres_layer_step", "attnres_synthetic_layer", "attnres_synthetic_layer_backward", "attnres_fold",
    "attnres_aggregate_fold",
    "attnres_linear", "attnres_linear_workspace_size", "attnres_linear_backward",
    "attnres_linear_backward_workspace_size", "attnres_qk_norm_rope", "attnres_qk_norm_rope_backward",
    "attnres_qk_norm_rope_backward_workspace_size", "attnres_linear_attention",
    "attnres_linear_attention_workspace_size", "attnres_linear_attention_backward",
    "attnres_linear_attention_backward_workspace_size", "attnres_linear_attention_step",
    "attnres_version", "AttnResState",
    "attnres_aggregate_host", "attnres_aggregate_host_workspace_size", "dtype_code", "AttnresError",
]

_DT = {torch.float32: ATTNRES_F32, torch.bfloat16: ATTNRES_BF16}


def dtype_code(dt: torch.dtype) -> int:
    try:
        return _DT[dt]
    except KeyError:
        raise TypeError(f"unsupported dtype {dt}; use float32 or bfloat16") from None


def _dev_ptr(t: torch.Tensor | None, name: str, dtype=None, contiguous=True) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    # the library launches on the current device: another device's memory
    # must never reach its kernels
    cur = torch.cuda.current_device()
    if t.get_device() != cur:
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{cur}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream) -> int:
    if stream is None:
        # the current stream's handle without building a Stream object
        if _RAW_STREAM is not None:
            return _RAW_STREAM(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def attnres_version() -> int:
    return _N.lib.attnres_version()


def attnres_num_sources(layer_idx: int, block_size: int, num_layers: int) -> int:
    """Sources of layer `layer_idx` (L+1 = the final output aggregation)."""
    return _N.check(_N.lib.attnres_num_sources(layer_idx, block_size, num_layers), "attnres_num_sources")


def attnres_aggregate(sources: Sequence[torch.Tensor] | torch.Tensor, w_l: torch.Tensor, out_r: torch.Tensor,
                      out_weights: torch.Tensor | None = None, eps: float = ATTNRES_DEFAULT_EPS,
                      dev_err: torch.Tensor | None = None, stream=None) -> None:
    """One layer of depth-wise attention.

    sources: S CUDA tensors [T, d] (float32 or bfloat16, one dtype), or one
    [S, T, d] tensor; w_l: [d] float32; out_r: [T, d] float32/bfloat16;
    out_weights: [T, S] float32 or None; dev_err: int32 [1] or None.
    """
    if isinstance(sources, torch.Tensor) and sources.dim() == 3 and not sources.is_contiguous():
        sources = list(sources.unbind(0))  # e.g. every other source: each slice checked below
    if isinstance(sources, torch.Tensor):
        # one contiguous [S, T, d] tensor: checked once, source s at base + s * T * d
        if sources.dim() != 3:
            raise ValueError("a stacked sources tensor must be [S, T, d]")
        S, T, d = sources.shape
        dt = sources.dtype
        base = _dev_ptr(sources, "sources")
        step = T * d * sources.element_size()
        ptrs = (ctypes.c_void_p * S)(*[base + i * step for i in range(S)]) if S else None
    else:
        srcs = list(sources)
        S = len(srcs)
        if not srcs:
            raise ValueError("need at least one source")
        T, d = srcs[0].shape
        dt = srcs[0].dtype
        for i, s in enumerate(srcs):
            if s.shape != (T, d) or s.dtype != dt:
                raise ValueError(f"source {i}: expected [{T}, {d}] {dt}, got {list(s.shape)} {s.dtype}")
        ptrs = (ctypes.c_void_p * S)(*[_dev_ptr(s, f"sources[{i}]") for i, s in enumerate(srcs)])
    if S < 1:
        raise ValueError("need at least one source")
    if out_r.shape != (T, d):
        raise ValueError("out_r must be [T, d]")
    if out_weights is not None and out_weights.shape != (T, S):
        raise ValueError("out_weights must be [T, S]")
    rc = _N.lib.attnres_aggregate(
        ptrs, S, T, d, dtype_code(dt), _dev_ptr(w_l, "w_l", torch.float32), float(eps),
        _dev_ptr(out_r, "out_r"), dtype_code(out_r.dtype), _dev_ptr(out_weights, "out_weights", torch.float32),
        _dev_ptr(dev_err, "dev_err", torch.int32), _stream_ptr(stream))
    _N.check(rc, "attnres_aggregate")


def attnres_aggregate_backward_workspace_size(T: int, d: int) -> int:
    """Bytes of device workspace attnres_aggregate_backward needs."""
    return _N.check(_N.lib.attnres_aggregate_backward_workspace_size(T, d), "attnres_aggregate_backward_workspace_size")


def attnres_aggregate_backward(sources: Sequence[torch.Tensor] | torch.Tensor, w_l: torch.Tensor,
                               grad_r: torch.Tensor, grad_sources: Sequence[torch.Tensor] | torch.Tensor,
                               grad_w: torch.Tensor, workspace: torch.Tensor | None = None,
                               eps: float = ATTNRES_DEFAULT_EPS, accumulate: bool = False,
                               dev_err: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of attnres_aggregate with respect to its sources and w_l
    (the forward is recomputed).  grad_sources: S tensors [T, d] (or one
    [S, T, d]) of the sources' dtype, overwritten or (accumulate) added to;
    grad_w: [d] float32, overwritten.  workspace: a device buffer of at least
    attnres_aggregate_backward_workspace_size(T, d) bytes (allocated here
    through torch when None)."""
    srcs = list(sources.unbind(0)) if isinstance(sources, torch.Tensor) else list(sources)
    grads = list(grad_sources.unbind(0)) if isinstance(grad_sources, torch.Tensor) else list(grad_sources)
    if len(grads) != len(srcs):
        raise ValueError("need one gradient buffer per source")
    T, d = srcs[0].shape
    dt = srcs[0].dtype
    for i, t in enumerate(srcs + grads + [grad_r]):
        if t.shape != (T, d) or t.dtype != dt:
            raise ValueError(f"tensor {i}: expected [{T}, {d}] {dt}")
    if workspace is None:
        nbytes = attnres_aggregate_backward_workspace_size(T, d)
        workspace = torch.empty(max(1, nbytes // 4), dtype=torch.float32, device=srcs[0].device)
    S = len(srcs)
    sp = (ctypes.c_void_p * S)(*[_dev_ptr(t, f"sources[{i}]") for i, t in enumerate(srcs)])
    gp = (ctypes.c_void_p * S)(*[_dev_ptr(t, f"grad_sources[{i}]") for i, t in enumerate(grads)])
    rc = _N.lib.attnres_aggregate_backward(
        sp, S, T, d, dtype_code(dt), _dev_ptr(w_l, "w_l", torch.float32), float(eps), _dev_ptr(grad_r, "grad_r"),
        gp, int(bool(accumulate)), _dev_ptr(grad_w, "grad_w", torch.float32), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _dev_ptr(dev_err, "dev_err", torch.int32), _stream_ptr(stream))
    _N.check(rc, "attnres_aggregate_backward")


def attnres_interblock_workspace_size(n: int, T: int, d: int, dtype: torch.dtype, Q: int) -> int:
    """Bytes of workspace attnres_interblock's tensor-core logits need (0: the
    path does not apply, e.g. fp32 sources)."""
    return _N.check(_N.lib.attnres_interblock_workspace_size(int(n), int(T), int(d), dtype_code(dtype), int(Q)),
                    "attnres_interblock_workspace_size")


def attnres_interblock(sources: Sequence[torch.Tensor], w_queries: Sequence[torch.Tensor] | torch.Tensor,
                       out_r: torch.Tensor, out_lse: torch.Tensor, out_weights: torch.Tensor | None = None,
                       eps: float = ATTNRES_DEFAULT_EPS, workspace: torch.Tensor | None = None,
                       tensor_cores: bool = True, dev_err: torch.Tensor | None = None, stream=None,
                       out_r0: torch.Tensor | None = None, out_weights0: torch.Tensor | None = None) -> None:
    """Phase 1 of the two-phase schedule: the n cached sources aggregated for
    Q queries at once.  out_r [Q, T, d] fp32, out_lse [Q, T] fp32,
    out_weights [Q, T, n] fp32 or None.  With tensor_cores (bf16 sources, d
    a multiple of 64) the logits run on the tensor cores in a workspace of
    attnres_interblock_workspace_size bytes (allocated here through torch
    when None); tensor_cores=False keeps every step on the CUDA cores.
    out_r0 [T, d] of the sources' dtype and out_weights0 [T, n] fp32 (or
    None): the block's first layer's output and weights, written here."""
    srcs = list(sources)
    qs = list(w_queries.unbind(0)) if isinstance(w_queries, torch.Tensor) else list(w_queries)
    T, d = srcs[0].shape
    dt = srcs[0].dtype
    ws_ptr, ws_bytes = None, 0
    if tensor_cores:
        need = attnres_interblock_workspace_size(len(srcs), T, d, dt, len(qs))
        if need > 0:
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=srcs[0].device)
            ws_ptr = _dev_ptr(workspace, "workspace")
            ws_bytes = workspace.numel() * workspace.element_size()
    sp = (ctypes.c_void_p * len(srcs))(*[_dev_ptr(t, f"sources[{i}]") for i, t in enumerate(srcs)])
    qp = (ctypes.c_void_p * len(qs))(*[_dev_ptr(q, f"w_queries[{i}]", torch.float32) for i, q in enumerate(qs)])
    rc = _N.lib.attnres_interblock(sp, len(srcs), T, d, dtype_code(dt), qp, len(qs), float(eps),
                                   _dev_ptr(out_r, "out_r", torch.float32), _dev_ptr(out_lse, "out_lse", torch.float32),
                                   _dev_ptr(out_weights, "out_weights", torch.float32),
                                   _dev_ptr(out_r0, "out_r0", dt), _dev_ptr(out_weights0, "out_weights0", torch.float32),
                                   ws_ptr, ws_bytes, _dev_ptr(dev_err, "dev_err", torch.int32), _stream_ptr(stream))
    _N.check(rc, "attnres_interblock")


def attnres_intrablock_step(state: "AttnResState", F_prev: torch.Tensor | None, w_l: torch.Tensor, layer_idx: int,
                            r_inter: torch.Tensor, lse_inter: torch.Tensor, a_inter: torch.Tensor | None,
                            out_r: torch.Tensor, out_weights: torch.Tensor | None = None,
                            dev_err: torch.Tensor | None = None, stream=None) -> None:
    """Phase 2 of the two-phase schedule for one layer (see include/attnres.h)."""
    rc = _N.lib.attnres_intrablock_step(
        ctypes.byref(state.struct), _dev_ptr(F_prev, "F_prev", state.h0.dtype), _dev_ptr(w_l, "w_l", torch.float32),
        layer_idx, _dev_ptr(r_inter, "r_inter", torch.float32), _dev_ptr(lse_inter, "lse_inter", torch.float32),
        _dev_ptr(a_inter, "a_inter", torch.float32), _dev_ptr(out_r, "out_r", state.h0.dtype),
        _dev_ptr(out_weights, "out_weights", torch.float32), _dev_ptr(dev_err, "dev_err", torch.int32),
        _stream_ptr(stream))
    _N.check(rc, "attnres_intrablock_step")


class AttnResState:
    """Resident depth sources of one batch (embedding, block sums, partial).

    Holds the torch buffers (so they outlive the C struct's pointers) and the
    `attnres_state` struct the C ABI updates.
    """

    def __init__(self, h0: torch.Tensor, block_reps: Sequence[torch.Tensor], partial: torch.Tensor,
                 num_layers: int, block_size: int, eps: float = ATTNRES_DEFAULT_EPS, early_loads: bool = False):
        T, d = h0.shape
        for i, b in enumerate(list(block_reps) + [partial]):
            if b.shape != (T, d) or b.dtype != h0.dtype:
                raise ValueError(f"state buffer {i} must be [{T}, {d}] {h0.dtype}")
        self.h0, self.block_reps, self.partial = h0, list(block_reps), partial
        self.num_layers, self.block_size = num_layers, block_size
        self.struct = _N.AttnresState()
        reps = (ctypes.c_void_p * max(1, len(self.block_reps)))(
            *[_dev_ptr(b, f"block_reps[{i}]") for i, b in enumerate(self.block_reps)])
        rc = _N.lib.attnres_state_init(ctypes.byref(self.struct), _dev_ptr(h0, "h0"), reps, len(self.block_reps),
                                       _dev_ptr(partial, "partial"), T, d, dtype_code(h0.dtype), num_layers,
                                       block_size, float(eps))
        _N.check(rc, "attnres_state_init")
        # ATTNRES_STATE_EARLY_LOADS: see include/attnres.h for when it is safe
        self.struct.flags = ATTNRES_STATE_EARLY_LOADS if early_loads else 0

    @classmethod
    def allocate(cls, h0: torch.Tensor, num_layers: int, block_size: int, eps: float = ATTNRES_DEFAULT_EPS,
                 early_loads: bool = False):
        n_blocks = -(-num_layers // block_size)
        reps = [torch.empty_like(h0) for _ in range(n_blocks)]
        return cls(h0, reps, torch.empty_like(h0), num_layers, block_size, eps, early_loads)

    @property
    def folded(self) -> int:
        return self.struct.folded

    def reset(self) -> None:
        _N.check(_N.lib.attnres_state_reset(ctypes.byref(self.struct)), "attnres_state_reset")

    def resume(self, folded: int) -> None:
        """Take up the stack after layer `folded` (v_1 .. v_folded already in
        the buffers, e.g. received at a pipeline stage boundary); see
        attnres_state_resume."""
        _N.check(_N.lib.attnres_state_resume(ctypes.byref(self.struct), int(folded)), "attnres_state_resume")


def attnres_layer_sources(state: AttnResState, layer_idx: int) -> list[int]:
    """Device pointers of layer `layer_idx`'s sources, in order."""
    out = (ctypes.c_void_p * ATTNRES_MAX_SOURCES)()
    n = ctypes.c_int(0)
    _N.check(_N.lib.attnres_layer_sources(ctypes.byref(state.struct), layer_idx, out, ctypes.byref(n)),
             "attnres_layer_sources")
    return [out[i] for i in range(n.value)]


def attnres_block_step(state: AttnResState, F_out: torch.Tensor, layer_idx: int,
                       dev_err: torch.Tensor | None = None, stream=None) -> None:
    """Fold layer `layer_idx`'s output into the partial sum / block representation."""
    rc = _N.lib.attnres_block_step(ctypes.byref(state.struct), _dev_ptr(F_out, "F_out", state.h0.dtype), layer_idx,
                                   _dev_ptr(dev_err, "dev_err", torch.int32), _stream_ptr(stream))
    _N.check(rc, "attnres_block_step")


def attnres_layer_step(state: AttnResState, F_prev: torch.Tensor | None, w_l: torch.Tensor, layer_idx: int,
                       out_r: torch.Tensor, out_weights: torch.Tensor | None = None,
                       dev_err: torch.Tensor | None = None, stream=None) -> None:
    """Fused: fold F_prev = v_{l-1}, then aggregate layer `layer_idx`.
    F_prev None: nothing left to fold (layer 1, or a resumed state)."""
    rc = _N.lib.attnres_layer_step(
        ctypes.byref(state.struct), _dev_ptr(F_prev, "F_prev", state.h0.dtype),
        _dev_ptr(w_l, "w_l", torch.float32), layer_idx, _dev_ptr(out_r, "out_r", state.h0.dtype),
        _dev_ptr(out_weights, "out_weights", torch.float32), _dev_ptr(dev_err, "dev_err", torch.int32),
        _stream_ptr(stream))
    _N.check(rc, "attnres_layer_step")


def attnres_synthetic_layer(x: torch.Tensor, g: torch.Tensor, s: torch.Tensor, out: torch.Tensor,
                            stream=None) -> None:
    """Stand-in layer body out = tanh(x * g) * s (drives a stack; not the method)."""
    T, d = x.shape
    rc = _N.lib.attnres_synthetic_layer(_dev_ptr(x, "x"), _dev_ptr(g, "g", torch.float32),
                                        _dev_ptr(s, "s", torch.float32), _dev_ptr(out, "out", x.dtype), T, d,
                                        dtype_code(x.dtype), _stream_ptr(stream))
    _N.check(rc, "attnres_synthetic_layer")


def attnres_synthetic_layer_backward(x: torch.Tensor, g: torch.Tensor, s: torch.Tensor, grad_out_a: torch.Tensor,
                                     grad_out_b: torch.Tensor | None, grad_x: torch.Tensor, stream=None) -> None:
    """Gradient of the stand-in body: grad_x = (grad_out_a + grad_out_b) * (1 - tanh(x g)^2) * g * s."""
    T, d = x.shape
    for name, t in (("grad_out_a", grad_out_a), ("grad_out_b", grad_out_b), ("grad_x", grad_x)):
        if t is not None and t.shape != (T, d):
            raise ValueError(f"{name} must be [T, d]")
    rc = _N.lib.attnres_synthetic_layer_backward(
        _dev_ptr(x, "x"), _dev_ptr(g, "g", torch.float32), _dev_ptr(s, "s", torch.float32),
        _dev_ptr(grad_out_a, "grad_out_a", x.dtype), _dev_ptr(grad_out_b, "grad_out_b", x.dtype),
        _dev_ptr(grad_x, "grad_x", x.dtype), T, d, dtype_code(x.dtype), _stream_ptr(stream))
    _N.check(rc, "attnres_synthetic_layer_backward")


def attnres_fold(prev: torch.Tensor | None, F: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Block bookkeeping on plain buffers: dst = prev + F (one rounding), or F when prev is None."""
    T, d = F.shape
    if dst.shape != (T, d) or (prev is not None and prev.shape != (T, d)):
        raise ValueError("prev, F and dst must all be [T, d]")
    rc = _N.lib.attnres_fold(_dev_ptr(prev, "prev", F.dtype), _dev_ptr(F, "F"), _dev_ptr(dst, "dst", F.dtype), T, d,
                             dtype_code(F.dtype), _stream_ptr(stream))
    _N.check(rc, "attnres_fold")


def attnres_aggregate_fold(sources: Sequence[torch.Tensor], prev: torch.Tensor | None, F: torch.Tensor,
                           dst: torch.Tensor, w_l: torch.Tensor, out_r: torch.Tensor,
                           out_weights: torch.Tensor | None = None, eps: float = ATTNRES_DEFAULT_EPS,
                           early_loads: bool = False, dev_err: torch.Tensor | None = None, stream=None) -> None:
    """One layer over the stored sources and the partial sum dst = prev + F
    (or F) formed and stored in the same launch; see include/attnres.h.
    Every row [T, d] of F's dtype; out_r the same; out_weights
    [T, len(sources) + 1] float32 or None.  early_loads: see
    ATTNRES_STATE_EARLY_LOADS (only when the kernel just before writes
    nothing this call reads but F)."""
    T, d = F.shape
    srcs = list(sources)
    for i, t in enumerate(srcs + [dst] + ([prev] if prev is not None else []) + [out_r]):
        if t.shape != (T, d) or t.dtype != F.dtype:
            raise ValueError(f"row {i}: expected [{T}, {d}] {F.dtype}, got {list(t.shape)} {t.dtype}")
    if out_weights is not None and out_weights.shape != (T, len(srcs) + 1):
        raise ValueError("out_weights must be [T, n_stored + 1]")
    ptrs = (ctypes.c_void_p * max(1, len(srcs)))(*[_dev_ptr(t, f"sources[{i}]") for i, t in enumerate(srcs)])
    rc = _N.lib.attnres_aggregate_fold(
        ptrs, len(srcs), _dev_ptr(prev, "prev"), _dev_ptr(F, "F"), _dev_ptr(dst, "dst"), T, d, dtype_code(F.dtype),
        _dev_ptr(w_l, "w_l", torch.float32), float(eps), _dev_ptr(out_r, "out_r"),
        _dev_ptr(out_weights, "out_weights", torch.float32), ATTNRES_STATE_EARLY_LOADS if early_loads else 0,
        _dev_ptr(dev_err, "dev_err", torch.int32), _stream_ptr(stream))
    _N.check(rc, "attnres_aggregate_fold")


def attnres_debug_wait_test(wait_limit_ns: int, withhold_row: int) -> None:
    """Diagnostic: make the ring kernels' bounded waits run out (withhold_row
    0..7 of every CTA's first token is armed without a copy; waits limited to
    wait_limit_ns).  (0, -1) restores normal operation."""
    _N.check(_N.lib.attnres_debug_wait_test(int(wait_limit_ns), int(withhold_row)), "attnres_debug_wait_test")


def _host_ptr(t: torch.Tensor | None, name: str, dtype=None) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise TypeError(f"{name} must be a CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def attnres_aggregate_host_workspace_size(S: int, chunk_tokens: int, d: int, src_dtype: torch.dtype,
                                          out_dtype: torch.dtype, with_weights: bool = True, slots: int = 2) -> int:
    """Bytes of device workspace attnres_aggregate_host needs for `slots`
    staging slots of chunk_tokens tokens."""
    return _N.check(_N.lib.attnres_aggregate_host_workspace_size(
        int(S), int(chunk_tokens), int(d), dtype_code(src_dtype), dtype_code(out_dtype), int(bool(with_weights)),
        int(slots)), "attnres_aggregate_host_workspace_size")


def attnres_aggregate_host(sources_host: Sequence[torch.Tensor] | torch.Tensor, w_host: torch.Tensor,
                           r_host: torch.Tensor, weights_host: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, chunk_tokens: int = 1024,
                           eps: float = ATTNRES_DEFAULT_EPS, dev_err: torch.Tensor | None = None,
                           stream=None) -> None:
    """attnres_aggregate with sources, query and outputs in host memory.

    sources_host: S CPU tensors [T, d] (float32 or bfloat16, one dtype,
    pinned for full speed) or one [S, T, d] CPU tensor; w_host: [d] float32;
    r_host: [T, d] float32/bfloat16; weights_host: [T, S] float32 or None;
    workspace: a CUDA tensor of at least attnres_aggregate_host_workspace_size
    bytes (None: two slots are allocated through torch).  The library streams
    token chunks through the workspace's staging slots; synchronise `stream`
    (default: the current stream) before reading r_host.
    """
    if isinstance(sources_host, torch.Tensor):
        if sources_host.dim() != 3:
            raise ValueError("a stacked sources tensor must be [S, T, d]")
        srcs = list(sources_host.unbind(0))
    else:
        srcs = list(sources_host)
    if not srcs:
        raise ValueError("need at least one source")
    T, d = srcs[0].shape
    dt = srcs[0].dtype
    for i, s in enumerate(srcs):
        if s.shape != (T, d) or s.dtype != dt:
            raise ValueError(f"source {i}: expected [{T}, {d}] {dt}, got {list(s.shape)} {s.dtype}")
    ptrs = (ctypes.c_void_p * len(srcs))(*[_host_ptr(s, f"sources_host[{i}]") for i, s in enumerate(srcs)])
    if r_host.shape != (T, d):
        raise ValueError("r_host must be [T, d]")
    if weights_host is not None and weights_host.shape != (T, len(srcs)):
        raise ValueError("weights_host must be [T, S]")
    if w_host.shape != (d,):
        raise ValueError("w_host must be [d]")
    if workspace is None:
        nbytes = attnres_aggregate_host_workspace_size(len(srcs), max(1, min(int(chunk_tokens), T)), d, dt,
                                                       r_host.dtype, weights_host is not None, 2)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=torch.cuda.current_device())
    rc = _N.lib.attnres_aggregate_host(
        ptrs, len(srcs), T, d, dtype_code(dt), _host_ptr(w_host, "w_host", torch.float32), float(eps),
        _host_ptr(r_host, "r_host"), dtype_code(r_host.dtype), _host_ptr(weights_host, "weights_host", torch.float32),
        int(chunk_tokens), _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _dev_ptr(dev_err, "dev_err", torch.int32), _stream_ptr(stream))
    _N.check(rc, "attnres_aggregate_host")


# ------------------------------------------------- operators of a layer body --

_ACT = {"none": ATTNRES_ACT_NONE, "gelu": ATTNRES_ACT_GELU, "gelu_tanh": ATTNRES_ACT_GELU_TANH,
        "silu": ATTNRES_ACT_SILU}


def activation_code(activation: str) -> int:
    try:
        return _ACT[activation]
    except KeyError:
        raise ValueError(f"unknown activation {activation!r}; use one of {sorted(_ACT)}") from None


_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_of(t, name: str) -> int:
    """The current device, on which a call's first tensor has to be."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0 or dev != _get_device():
        _dev_ptr(t, name, contiguous=False)
    return dev


def _stream_on(stream, cur: int) -> int:
    """_stream_ptr where the current device is known."""
    return _RAW_STREAM(cur) if stream is None and _RAW_STREAM is not None else _stream_ptr(stream)


def _where(t, name: str, dtype: torch.dtype, cur: int) -> None:
    """Say what is wrong with a tensor that is not of `dtype` on device `cur`."""
    _dev_ptr(t, name, dtype, contiguous=False)
    raise ValueError(f"{name} is on {t.device} but the current device is cuda:{cur}")


def _rows(t: torch.Tensor | None, name: str, shape: tuple, dtype: torch.dtype, cur: int) -> tuple[int | None, int]:
    """Pointer and row stride (elements) of a tensor on device `cur` whose
    rows (everything behind the first dimension) are contiguous; None:
    (None, row length)."""
    width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    if t is None:
        return None, width
    if not isinstance(t, torch.Tensor) or t.get_device() != cur or t.dtype is not dtype:
        _where(t, name, dtype, cur)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), width
    st, last = t.stride(), shape[-1]
    if (st[-1] != 1 and last > 1) or (len(shape) == 3 and st[1] != last and shape[1] > 1):
        raise ValueError(f"the rows of {name} must be contiguous")
    if shape[0] > 1 and st[0] < width:
        raise ValueError(f"the rows of {name} overlap")
    return t.data_ptr(), st[0] if shape[0] > 1 else width


def _vec(t: torch.Tensor | None, name: str, shape: tuple, dtype: torch.dtype, cur: int) -> int | None:
    """Pointer of a contiguous tensor on device `cur`."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != cur or t.dtype is not dtype:
        _where(t, name, dtype, cur)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _workspace(workspace: torch.Tensor | None, nbytes: int, device, stream) -> tuple[torch.Tensor | None, int | None, int]:
    """The caller's workspace, or one allocated through torch for the stream
    the call runs on (so that torch does not hand it out again while the
    kernels use it).  (tensor to keep, pointer, bytes)."""
    if workspace is None:
        if nbytes <= 0:
            return None, None, 0
        if stream is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            with torch.cuda.stream(s):
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), nbytes
    return workspace, _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()


def _matrix(t: torch.Tensor, name: str) -> tuple[int, int]:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-d tensor")
    return t.shape[0], t.shape[1]


def _place(t: torch.Tensor | None, cols: int) -> tuple[int | None, int]:
    """Address and row stride of an operand ([rows, cols]; None: aligned rows)."""
    return (None, cols) if t is None else (t.data_ptr(), t.stride(0) if t.shape[0] > 1 else cols)


def attnres_linear_workspace_size(M: int, N: int, K: int, dtype: torch.dtype, x: torch.Tensor | None = None,
                                  w: torch.Tensor | None = None) -> int:
    """Bytes of device workspace with which attnres_linear takes its fastest
    path for contiguous operands of these sizes; given x or w, for these ones
    (bf16 rows off the 16-byte boundaries are copied)."""
    return _N.check(_N.lib.attnres_linear_operands_workspace_size(*_place(x, K), _place(w, K)[0], M, N, K, dtype_code(dtype)),
                    "attnres_linear_workspace_size")


def attnres_linear(x: torch.Tensor, w: torch.Tensor, out: torch.Tensor, bias: torch.Tensor | None = None,
                   residual: torch.Tensor | None = None, activation: str = "none",
                   workspace: torch.Tensor | None = None, dev_err: torch.Tensor | None = None, stream=None) -> None:
    """out = act(x w^T + bias) + residual.

    x: [M, K]; w: [N, K]; out, residual: [M, N], all float32 or all bfloat16
    (rows contiguous, w wholly); bias: [N] float32; residual may be out
    itself.  activation: "none", "gelu", "gelu_tanh" or "silu".  workspace:
    a device buffer of attnres_linear_workspace_size bytes (allocated here
    through torch when None, with room for the operands as they lie).
    """
    M, K = _matrix(x, "x")
    N = _matrix(w, "w")[0]
    dt = x.dtype
    code = dtype_code(dt)
    act = activation_code(activation)
    cur = _device_of(x, "x")
    xp, ldx = _rows(x, "x", (M, K), dt, cur)
    wp = _vec(w, "w", (N, K), dt, cur)
    op, ldo = _rows(out, "out", (M, N), dt, cur)
    rp, ldr = _rows(residual, "residual", (M, N), dt, cur)
    need = 0
    if workspace is None:
        need = _N.check(_N.lib.attnres_linear_operands_workspace_size(xp, ldx, wp, M, N, K, code), "attnres_linear_workspace_size")
    _keep, ws, nbytes = _workspace(workspace, need, x.device, stream)
    rc = _N.lib.attnres_linear(xp, ldx, wp, _vec(bias, "bias", (N,), torch.float32, cur), rp, ldr, op, ldo, M, N, K, code, act,
                               ws, nbytes, _dev_ptr(dev_err, "dev_err", torch.int32), _stream_on(stream, cur))
    _N.check(rc, "attnres_linear")


def attnres_linear_backward_workspace_size(M: int, N: int, K: int, dtype: torch.dtype, activation: str = "none",
                                           x: torch.Tensor | None = None, w: torch.Tensor | None = None,
                                           grad_out: torch.Tensor | None = None) -> int:
    """Bytes of device workspace attnres_linear_backward needs; given operands,
    with room for the copies of those off the 16-byte boundaries."""
    return _N.check(_N.lib.attnres_linear_backward_operands_workspace_size(
        *_place(x, K), _place(w, K)[0], *_place(grad_out, N), M, N, K, dtype_code(dtype), activation_code(activation)),
        "attnres_linear_backward_workspace_size")


def attnres_linear_backward(x: torch.Tensor, w: torch.Tensor, grad_out: torch.Tensor,
                            grad_x: torch.Tensor | None = None, grad_w: torch.Tensor | None = None,
                            grad_bias: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                            activation: str = "none", workspace: torch.Tensor | None = None,
                            dev_err: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of attnres_linear with respect to x, w and bias (those not
    None are overwritten); the residual's gradient is grad_out.  grad_x
    [M, K], grad_w [N, K] of x's dtype, grad_bias [N] float32."""
    M, K = _matrix(x, "x")
    N = _matrix(w, "w")[0]
    dt = x.dtype
    code = dtype_code(dt)
    act = activation_code(activation)
    cur = _device_of(x, "x")
    xp, ldx = _rows(x, "x", (M, K), dt, cur)
    wp = _vec(w, "w", (N, K), dt, cur)
    gp, ldg = _rows(grad_out, "grad_out", (M, N), dt, cur)
    need = 0
    if workspace is None:
        need = _N.check(_N.lib.attnres_linear_backward_operands_workspace_size(xp, ldx, wp, gp, ldg, M, N, K, code, act),
                        "attnres_linear_backward_workspace_size")
    _keep, ws, nbytes = _workspace(workspace, need, x.device, stream)
    rc = _N.lib.attnres_linear_backward(
        xp, ldx, wp, _vec(bias, "bias", (N,), torch.float32, cur), gp, ldg, _vec(grad_x, "grad_x", (M, K), dt, cur),
        _vec(grad_w, "grad_w", (N, K), dt, cur), _vec(grad_bias, "grad_bias", (N,), torch.float32, cur), M, N, K, code, act, ws,
        nbytes, _dev_ptr(dev_err, "dev_err", torch.int32), _stream_on(stream, cur))
    _N.check(rc, "attnres_linear_backward")


def _heads(t: torch.Tensor | None, name: str) -> tuple[int, int, int]:
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, channels]")
    return tuple(t.shape)


def _qk_sizes(q, k, positions, inv_freq):
    """(T, D, dtype, Hq, Hk) of a q and a k, either of them None."""
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq come together")
    first = q if q is not None else k
    T, _, D = _heads(first, "q" if q is not None else "k")
    return T, D, first.dtype, q.shape[1] if q is not None else 0, _heads(k, "k")[1] if k is not None else 0


def _rope_args(T: int, positions, inv_freq, interleaved: bool, cur: int):
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    return (_vec(positions, "positions", (T,), torch.int64, cur),
            _vec(inv_freq, "inv_freq", (rot // 2,), torch.float32, cur), rot, int(bool(interleaved)))


def attnres_qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, q_out: torch.Tensor | None,
                         k_out: torch.Tensor | None, q_gain: torch.Tensor | None = None,
                         k_gain: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                         inv_freq: torch.Tensor | None = None, interleaved: bool = False,
                         eps: float = ATTNRES_DEFAULT_EPS, stream=None) -> None:
    """RMSNorm of every head of q [T, Hq, D] and k [T, Hk, D] (either may be
    None) with gains [D] float32 or None, and rotation of the first
    2 len(inv_freq) channels by positions [T] int64 times inv_freq float32
    (both None: no rotation).  Heads and channels contiguous, tokens at any
    stride; q_out may be q and k_out k."""
    T, D, dt, Hq, Hk = _qk_sizes(q, k, positions, inv_freq)
    code = dtype_code(dt)
    cur = _device_of(q if q is not None else k, "q" if q is not None else "k")
    pos, freq, rot, inter = _rope_args(T, positions, inv_freq, interleaved, cur)
    qp, qs = _rows(q, "q", (T, Hq, D), dt, cur)
    kp, ks = _rows(k, "k", (T, Hk, D), dt, cur)
    qo, qos = _rows(q_out if q is not None else None, "q_out", (T, Hq, D), dt, cur)
    ko, kos = _rows(k_out if k is not None else None, "k_out", (T, Hk, D), dt, cur)
    rc = _N.lib.attnres_qk_norm_rope(qp, qs, Hq, kp, ks, Hk, T, D, code, _vec(q_gain, "q_gain", (D,), torch.float32, cur),
                                     _vec(k_gain, "k_gain", (D,), torch.float32, cur), float(eps), pos, freq, rot, inter,
                                     qo, qos, ko, kos, _stream_on(stream, cur))
    _N.check(rc, "attnres_qk_norm_rope")


def attnres_qk_norm_rope_backward_workspace_size(T: int, Hq: int, Hk: int, D: int) -> int:
    """Bytes of device workspace the gain gradients of attnres_qk_norm_rope_backward need."""
    return _N.check(_N.lib.attnres_qk_norm_rope_backward_workspace_size(T, Hq, Hk, D),
                    "attnres_qk_norm_rope_backward_workspace_size")


def attnres_qk_norm_rope_backward(q: torch.Tensor | None, k: torch.Tensor | None, grad_q_out: torch.Tensor | None,
                                  grad_k_out: torch.Tensor | None, grad_q: torch.Tensor | None,
                                  grad_k: torch.Tensor | None, q_gain: torch.Tensor | None = None,
                                  k_gain: torch.Tensor | None = None, grad_q_gain: torch.Tensor | None = None,
                                  grad_k_gain: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                                  inv_freq: torch.Tensor | None = None, interleaved: bool = False,
                                  eps: float = ATTNRES_DEFAULT_EPS, workspace: torch.Tensor | None = None,
                                  stream=None) -> None:
    """Gradients of attnres_qk_norm_rope, from the forward's inputs (q and k
    as they were before it).  grad_q may be grad_q_out and grad_k grad_k_out;
    the gain gradients ([D] float32) are overwritten, or skipped when None."""
    T, D, dt, Hq, Hk = _qk_sizes(q, k, positions, inv_freq)
    code = dtype_code(dt)
    cur = _device_of(q if q is not None else k, "q" if q is not None else "k")
    pos, freq, rot, inter = _rope_args(T, positions, inv_freq, interleaved, cur)
    qp, qs = _rows(q, "q", (T, Hq, D), dt, cur)
    kp, ks = _rows(k, "k", (T, Hk, D), dt, cur)
    gqo, gqos = _rows(grad_q_out if q is not None else None, "grad_q_out", (T, Hq, D), dt, cur)
    gko, gkos = _rows(grad_k_out if k is not None else None, "grad_k_out", (T, Hk, D), dt, cur)
    gq, gqs = _rows(grad_q if q is not None else None, "grad_q", (T, Hq, D), dt, cur)
    gk, gks = _rows(grad_k if k is not None else None, "grad_k", (T, Hk, D), dt, cur)
    dgq = _vec(grad_q_gain, "grad_q_gain", (D,), torch.float32, cur)
    dgk = _vec(grad_k_gain, "grad_k_gain", (D,), torch.float32, cur)
    need = 0
    if workspace is None and (dgq is not None or dgk is not None):
        need = attnres_qk_norm_rope_backward_workspace_size(T, Hq, Hk, D)
    _keep, ws, nbytes = _workspace(workspace, need, (q if q is not None else k).device, stream)
    rc = _N.lib.attnres_qk_norm_rope_backward(
        qp, qs, Hq, kp, ks, Hk, T, D, code, _vec(q_gain, "q_gain", (D,), torch.float32, cur),
        _vec(k_gain, "k_gain", (D,), torch.float32, cur), float(eps), pos, freq, rot, inter, gqo, gqos, gko, gkos, gq, gqs,
        gk, gks, dgq, dgk, ws, nbytes, _stream_on(stream, cur))
    _N.check(rc, "attnres_qk_norm_rope_backward")


def _attention_args(q, k, v, log_decay, cu_seqlens, cur: int):
    T, H, Dk = _heads(q, "q")
    Dv = _heads(v, "v")[2]
    dt = q.dtype
    code = dtype_code(dt)
    qp, qs = _rows(q, "q", (T, H, Dk), dt, cur)
    kp, ks = _rows(k, "k", (T, H, Dk), dt, cur)
    vp, vs = _rows(v, "v", (T, H, Dv), dt, cur)
    if isinstance(log_decay, torch.Tensor) and log_decay.requires_grad:
        raise ValueError("log_decay is a constant: it gets no gradient")
    g = _vec(log_decay, "log_decay", (H,), torch.float32, cur)
    N = 1
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        if N < 1:
            raise ValueError("cu_seqlens must hold at least two offsets")
    cu = _vec(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, cur)
    return T, H, Dk, Dv, dt, (qp, qs, kp, ks, vp, vs, T, H, Dk, Dv, code, g), cu, N


def attnres_linear_attention_workspace_size(T: int, H: int, Dk: int, Dv: int, dtype: torch.dtype, num_seqs: int = 1) -> int:
    """Bytes of device workspace that attnres_linear_attention needs for up to T
    tokens in up to num_seqs sequences (0: none)."""
    return _N.check(_N.lib.attnres_linear_attention_workspace_size(T, H, Dk, Dv, dtype_code(dtype), num_seqs),
                    "attnres_linear_attention_workspace_size")


def attnres_linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                             out: torch.Tensor, cu_seqlens: torch.Tensor | None = None,
                             initial_state: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
                             scale: float | None = None, workspace: torch.Tensor | None = None,
                             dev_err: torch.Tensor | None = None, stream=None) -> None:
    """Causal linear attention over prompts, S_t = e^log_decay S_{t-1} + k_t v_t^T,
    out_t = scale q_t S_t (scale None: 1/sqrt(Dk)).

    q, k: [T, H, Dk]; v, out: [T, H, Dv], float32 or bfloat16, tokens at any
    stride; log_decay: [H] float32; cu_seqlens: [num_seqs + 1] int32 on the
    device (None: one sequence); initial_state, final_state: [num_seqs, H,
    Dk, Dv] float32 or None, possibly the same tensor.
    """
    cur = _device_of(q, "q")
    T, H, Dk, Dv, dt, head, cu, N = _attention_args(q, k, v, log_decay, cu_seqlens, cur)
    op, os_ = _rows(out, "out", (T, H, Dv), dt, cur)
    shape = (N, H, Dk, Dv)
    s0 = _vec(initial_state, "initial_state", shape, torch.float32, cur)
    s1 = _vec(final_state, "final_state", shape, torch.float32, cur)
    need = 0 if workspace is not None else attnres_linear_attention_workspace_size(T, H, Dk, Dv, dt, N)
    _keep, ws, nbytes = _workspace(workspace, need, q.device, stream)
    rc = _N.lib.attnres_linear_attention(*head, cu, N, s0, s1, float(Dk ** -0.5 if scale is None else scale), op, os_,
                                         ws, nbytes, _dev_ptr(dev_err, "dev_err", torch.int32), _stream_on(stream, cur))
    _N.check(rc, "attnres_linear_attention")


def attnres_linear_attention_backward_workspace_size(T: int, H: int, Dk: int, Dv: int, dtype: torch.dtype,
                                                     num_seqs: int = 1) -> int:
    """Bytes of device workspace that attnres_linear_attention_backward needs for
    up to T tokens in up to num_seqs sequences (0: none)."""
    return _N.check(_N.lib.attnres_linear_attention_backward_workspace_size(T, H, Dk, Dv, dtype_code(dtype), num_seqs),
                    "attnres_linear_attention_backward_workspace_size")


def attnres_linear_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                                      grad_out: torch.Tensor, grad_q: torch.Tensor | None, grad_k: torch.Tensor | None,
                                      grad_v: torch.Tensor | None, cu_seqlens: torch.Tensor | None = None,
                                      initial_state: torch.Tensor | None = None,
                                      grad_final_state: torch.Tensor | None = None,
                                      grad_initial_state: torch.Tensor | None = None, scale: float | None = None,
                                      workspace: torch.Tensor | None = None, dev_err: torch.Tensor | None = None,
                                      stream=None) -> None:
    """Gradients of attnres_linear_attention from the forward's inputs
    (grad_q, grad_k, grad_v contiguous, of q's dtype; the states' float32).
    Those that are None are not formed; grad_initial_state comes with grad_v."""
    cur = _device_of(q, "q")
    T, H, Dk, Dv, dt, head, cu, N = _attention_args(q, k, v, log_decay, cu_seqlens, cur)
    gp, gs = _rows(grad_out, "grad_out", (T, H, Dv), dt, cur)
    shape = (N, H, Dk, Dv)
    s0 = _vec(initial_state, "initial_state", shape, torch.float32, cur)
    ds1 = _vec(grad_final_state, "grad_final_state", shape, torch.float32, cur)
    ds0 = _vec(grad_initial_state, "grad_initial_state", shape, torch.float32, cur)
    need = 0 if workspace is not None else attnres_linear_attention_backward_workspace_size(T, H, Dk, Dv, dt, N)
    _keep, ws, nbytes = _workspace(workspace, need, q.device, stream)
    rc = _N.lib.attnres_linear_attention_backward(
        *head, cu, N, s0, float(Dk ** -0.5 if scale is None else scale), gp, gs, ds1, _vec(grad_q, "grad_q", (T, H, Dk), dt, cur),
        _vec(grad_k, "grad_k", (T, H, Dk), dt, cur), _vec(grad_v, "grad_v", (T, H, Dv), dt, cur), ds0, ws, nbytes,
        _dev_ptr(dev_err, "dev_err", torch.int32), _stream_on(stream, cur))
    _N.check(rc, "attnres_linear_attention_backward")


def attnres_linear_attention_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                                  state: torch.Tensor, out: torch.Tensor, slots: torch.Tensor | None = None,
                                  scale: float | None = None, stream=None) -> None:
    """One token per row: state [num_slots, H, Dk, Dv] float32 of slot
    slots[b] (int32; None: b) updated in place, out [B, H, Dv] written.  A
    slot outside the pool marks a padding row (its out row stays); rows of
    one slot are consecutive tokens in row order."""
    cur = _device_of(q, "q")
    B, H, Dk, Dv, dt, head, _, _ = _attention_args(q, k, v, log_decay, None, cur)
    op, os_ = _rows(out, "out", (B, H, Dv), dt, cur)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be [num_slots, H, Dk, Dv]")
    num_slots = state.shape[0]
    sp = _vec(state, "state", (num_slots, H, Dk, Dv), torch.float32, cur)
    rc = _N.lib.attnres_linear_attention_step(*head, sp, num_slots, _vec(slots, "slots", (B,), torch.int32, cur),
                                              float(Dk ** -0.5 if scale is None else scale), op, os_,
                                              _stream_on(stream, cur))
    _N.check(rc, "attnres_linear_attention_step")
