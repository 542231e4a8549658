"""Argument checks of layer norm, gated recurrence and gradient clipping:
refused on the host, before any launch (no GPU needed; the pointers are never
dereferenced)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def N():
    import __graft_entry__
    B = __graft_entry__._build_module()
    if not os.path.exists(B.LIB_PATH):
        B.build()
    from depth_wise_attention_block_gb300 import _native
    return _native


X, F, G, OUT, WS, DY, V = (0x10000000 * (i + 1) for i in range(7))
FAR = 1 << 60


def _ln(N, **kw):
    a = dict(x=X, xs=64, T=10, d=64, dt=1, gain=V, bias=V + 4096, eps=1e-5, out=OUT, os=64)
    a.update(kw)
    return N.lib.attnres_layer_norm(*[a[n] for n in ("x", "xs", "T", "d", "dt", "gain", "bias", "eps", "out", "os")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), "EDTYPE"), (dict(T=-1), "EINVAL"), (dict(d=0), "EINVAL"), (dict(d=(1 << 24) + 1, xs=1 << 25, os=1 << 25), "ERANGE"),
    (dict(eps=-1.0), "EINVAL"), (dict(eps=float("nan")), "EINVAL"), (dict(eps=float("inf")), "EINVAL"), (dict(xs=63), "EINVAL"),
    (dict(os=63), "EINVAL"), (dict(xs=FAR), "EINVAL"), (dict(T=1 << 40, xs=64), "ERANGE"), (dict(T=1 << 40, os=64, xs=64), "ERANGE"),
    (dict(x=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(out=X + 2), "EINVAL"), (dict(out=X, os=128), "EINVAL"),
    (dict(out=V), "EINVAL"), (dict(out=V + 4096 + 252), "EINVAL"), (dict(x=X + 1), "EINVAL"), (dict(dt=0, out=OUT + 2), "EINVAL"),
])
def test_layer_norm_refuses(N, kw, code):
    assert _ln(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def _ln_bwd(N, **kw):
    a = dict(x=X, xs=64, T=10, d=64, dt=1, gain=V, eps=1e-5, dy=DY, dys=64, gx=OUT, gxs=64, gg=OUT + 0x100000, gb=OUT + 0x200000,
             ws=WS, wsb=1 << 24)
    a.update(kw)
    return N.lib.attnres_layer_norm_backward(*[a[n] for n in ("x", "xs", "T", "d", "dt", "gain", "eps", "dy", "dys", "gx", "gxs", "gg",
                                                             "gb", "ws", "wsb")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=-1), "EDTYPE"), (dict(x=None), "EINVAL"), (dict(dy=None), "EINVAL"), (dict(dys=63), "EINVAL"), (dict(gxs=63), "EINVAL"),
    (dict(ws=None), "EINVAL"), (dict(gx=X), "EINVAL"), (dict(gx=DY + 2), "EINVAL"), (dict(gx=DY, gxs=128), "EINVAL"), (dict(gg=V), "EINVAL"),
    (dict(gb=OUT), "EINVAL"), (dict(gb=OUT + 0x100000), "EINVAL"), (dict(dy=DY + 1), "EINVAL"), (dict(dt=0, gx=OUT + 2), "EINVAL"), (dict(ws=X - 256), "EINVAL"), (dict(ws=OUT), "EINVAL"),
])
def test_layer_norm_backward_refuses(N, kw, code):
    assert _ln_bwd(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def test_layer_norm_without_rows_or_gradients(N):
    assert _ln(N, T=0, x=None, out=None) == 0
    assert _ln_bwd(N, gx=None, gg=None, gb=None, ws=None, dy=None) == 0
    assert _ln_bwd(N, T=0, x=None, dy=None, gg=None, gb=None, ws=None) == 0
    assert N.lib.attnres_layer_norm_backward_workspace_size(-1, 4) == N.ATTNRES_EINVAL
    assert N.lib.attnres_layer_norm_backward_workspace_size(4, 0) == N.ATTNRES_EINVAL
    assert N.lib.attnres_layer_norm_backward_workspace_size(4, 1 << 25) == N.ATTNRES_ERANGE


def _gr(N, **kw):
    a = dict(x=X, xs=64, f=F, fs=64, g=G, gs=64, T=100, C=64, dt=1, cu=None, n=1, s0=None, s1=None, out=OUT, os=64, ch=None)
    a.update(kw)
    return N.lib.attnres_gated_recurrence(*[a[n] for n in ("x", "xs", "f", "fs", "g", "gs", "T", "C", "dt", "cu", "n", "s0", "s1", "out",
                                                          "os", "ch")], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), "EDTYPE"), (dict(T=-1), "EINVAL"), (dict(C=0), "EINVAL"), (dict(n=0), "EINVAL"), (dict(n=2), "EINVAL"),
    (dict(T=1 << 31), "ERANGE"), (dict(n=65536, cu=V), "ERANGE"), (dict(C=1 << 25, xs=1 << 26), "ERANGE"), (dict(x=None), "EINVAL"),
    (dict(f=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(xs=63), "EINVAL"), (dict(fs=63), "EINVAL"), (dict(gs=63), "EINVAL"),
    (dict(os=63), "EINVAL"), (dict(T=1 << 30, xs=1 << 20), "ERANGE"), (dict(out=X), "EINVAL"), (dict(out=F), "EINVAL"),
    (dict(out=G + 2), "EINVAL"), (dict(s0=V, s1=V + 4), "EINVAL"), (dict(s1=OUT), "EINVAL"), (dict(ch=OUT + 64), "EINVAL"),
    (dict(s1=V, ch=V), "EINVAL"), (dict(cu=V, s1=V), "EINVAL"), (dict(ch=X), "EINVAL"), (dict(x=X + 1), "EINVAL"), (dict(f=F + 1), "EINVAL"),
    (dict(g=G + 1), "EINVAL"), (dict(dt=0, out=OUT + 2), "EINVAL"),
])
def test_gated_recurrence_refuses(N, kw, code):
    assert _gr(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def _gr_bwd(N, **kw):
    a = dict(x=X, xs=64, f=F, fs=64, g=G, gs=64, T=100, C=64, dt=1, cu=None, n=1, s0=None, ch=V, dy=DY, dys=64, ds1=None, gx=OUT, gxs=64,
             gf=OUT + 0x100000, gfs=64, gg=OUT + 0x200000, ggs=64, ds0=None)
    a.update(kw)
    return N.lib.attnres_gated_recurrence_backward(*[a[n] for n in (
        "x", "xs", "f", "fs", "g", "gs", "T", "C", "dt", "cu", "n", "s0", "ch", "dy", "dys", "ds1", "gx", "gxs", "gf", "gfs", "gg", "ggs",
        "ds0")], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), "EDTYPE"), (dict(dy=None), "EINVAL"), (dict(ch=None), "EINVAL"), (dict(g=None), "EINVAL"), (dict(dys=63), "EINVAL"),
    (dict(gxs=63), "EINVAL"), (dict(gfs=63), "EINVAL"), (dict(ggs=63), "EINVAL"), (dict(gx=X), "EINVAL"), (dict(gf=F), "EINVAL"),
    (dict(gx=DY), "EINVAL"), (dict(gf=OUT), "EINVAL"), (dict(gg=OUT + 0x100000 + 2), "EINVAL"), (dict(gx=V), "EINVAL"),
    (dict(ds0=OUT), "EINVAL"), (dict(ds0=WS, ds1=WS + 4), "EINVAL"), (dict(s0=WS, ds0=WS), "EINVAL"), (dict(n=3), "EINVAL"),
])
def test_gated_recurrence_backward_refuses(N, kw, code):
    assert _gr_bwd(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def _step(N, **kw):
    a = dict(x=X, xs=64, f=F, fs=64, g=G, gs=64, B=9, C=64, dt=1, st=WS, ns=9, slots=None, out=OUT, os=64)
    a.update(kw)
    return N.lib.attnres_gated_recurrence_step(*[a[n] for n in ("x", "xs", "f", "fs", "g", "gs", "B", "C", "dt", "st", "ns", "slots", "out",
                                                               "os")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "EINVAL"), (dict(B=65536), "ERANGE"), (dict(ns=8), "EINVAL"), (dict(ns=-1), "EINVAL"), (dict(st=None), "EINVAL"),
    (dict(out=None), "EINVAL"), (dict(st=X), "EINVAL"), (dict(out=F), "EINVAL"), (dict(st=OUT), "EINVAL"), (dict(dt=9), "EDTYPE"),
    (dict(os=63), "EINVAL"), (dict(slots=OUT), "EINVAL"),
])
def test_step_refuses(N, kw, code):
    assert _step(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


@pytest.mark.parametrize("call,kw", [
    (_ln, dict(gain=V + 2)), (_ln, dict(bias=V + 4098)), (_ln_bwd, dict(gain=V + 2)), (_ln_bwd, dict(gg=V + 0x10001)),
    (_ln_bwd, dict(gb=V + 0x10003)), (_gr, dict(cu=V + 1)), (_gr, dict(s0=V + 2)), (_gr, dict(s1=V + 2)), (_gr, dict(ch=V + 2)),
    (_gr_bwd, dict(ch=V + 2)), (_gr_bwd, dict(ds1=WS + 2)), (_gr_bwd, dict(ds0=WS + 1)), (_step, dict(st=WS + 2)),
    (_step, dict(slots=V + 2)),
])
def test_float_and_int32_arrays_off_their_words(N, call, kw):
    assert call(N, **kw) == N.ATTNRES_EINVAL
    assert b"4-byte" in N.lib.attnres_last_error()


def test_recurrence_without_rows(N):
    assert _gr(N, T=0, x=None, f=None, g=None, out=None) == 0
    assert _gr_bwd(N, gx=None, gf=None, gg=None, dy=None, ch=None) == 0
    assert _gr_bwd(N, T=0, x=None, f=None, g=None, gg=None, dy=None, ch=None) == 0
    assert _step(N, B=0, x=None, f=None, g=None, out=None, st=None) == 0
    assert _step(N, ns=0, slots=V) == 0


def _clip(N, ptrs=(X, F), outs=(X, F), sizes=(10, 20), dts=(1, 0), n=None, max_norm=1.0, norm=V, ws=WS, wsb=1 << 20):
    k = len(sizes)
    vp = lambda p: None if p is None else (ctypes.c_void_p * k)(*p)  # noqa: E731
    return N.lib.attnres_grad_clip(vp(ptrs), vp(outs), (ctypes.c_int64 * k)(*sizes), (ctypes.c_int * k)(*dts), k if n is None else n,
                                   max_norm, norm, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), "EINVAL"), (dict(n=65536), "ERANGE"), (dict(ptrs=None), "EINVAL"), (dict(dts=(1, 2)), "EDTYPE"),
    (dict(sizes=(10, -1)), "EINVAL"), (dict(sizes=(10, 1 << 43)), "ERANGE"), (dict(ptrs=(X, None)), "EINVAL"),
    (dict(outs=(X, None)), "EINVAL"), (dict(max_norm=-1.0), "EINVAL"), (dict(max_norm=float("nan")), "EINVAL"),
    (dict(norm=None), "EINVAL"), (dict(norm=V + 2), "EINVAL"), (dict(norm=X + 4), "EINVAL"), (dict(norm=F + 76, outs=(G, G + 4096)), "EINVAL"),
    (dict(outs=(X, X)), "EINVAL"), (dict(outs=(F, G)), "EINVAL"), (dict(outs=(X + 2, F)), "EINVAL"), (dict(outs=(G, G + 16)), "EINVAL"),
    (dict(ptrs=(X, X + 16), outs=(X, X + 16)), "EINVAL"), (dict(ptrs=(X, F + 2), outs=(X, F + 2)), "EINVAL"),
    (dict(ptrs=(X + 1, F), outs=(X + 1, F)), "EINVAL"), (dict(outs=(X, G + 1)), "EINVAL"), (dict(ws=X - 256, wsb=512), "EINVAL"),
    (dict(ws=V - 256, wsb=512), "EINVAL"),
])
def test_grad_clip_refuses(N, kw, code):
    assert _clip(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def test_python_checks(N):
    import torch
    import depth_wise_attention_block_gb300 as A
    from depth_wise_attention_block_gb300 import autograd as AG
    x = torch.zeros(2, 4)
    with pytest.raises(ValueError, match="2-d"):
        A.attnres_layer_norm(x[0], x)
    with pytest.raises(TypeError, match="dtype"):
        A.attnres_layer_norm(x.half(), x)
    with pytest.raises(TypeError, match="CUDA"):
        A.attnres_layer_norm(x, x)
    with pytest.raises(TypeError, match="CUDA"):
        A.attnres_layer_norm_backward(x, x, x)
    with pytest.raises(TypeError, match="CUDA"):
        A.attnres_gated_recurrence(x, x, x)
    with pytest.raises(TypeError, match="CUDA"):
        A.attnres_gated_recurrence_step(x, x, x, x)
    with pytest.raises(TypeError, match="CUDA"):
        A.attnres_grad_clip([x], 1.0, x[0, :1])
    with pytest.raises(ValueError, match="holds a gradient"):
        AG.clip_grad_norm([x], 1.0)
