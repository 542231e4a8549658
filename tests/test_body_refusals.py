"""Argument checks of the layer body's operators: refused on the host, before
any launch (no GPU needed; the pointers are never dereferenced)."""
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


X, W, BI, RE, OUT, WS = (0x10000000 * (i + 1) for i in range(6))


def _linear(lib, **kw):
    a = dict(x=X, ldx=64, w=W, bias=BI, res=RE, ldr=32, out=OUT, ldo=32, M=10, N=32, K=64, dt=1, act=0, ws=None, wsb=0)
    a.update(kw)
    return lib.lib.attnres_linear(a["x"], a["ldx"], a["w"], a["bias"], a["res"], a["ldr"], a["out"], a["ldo"], a["M"], a["N"],
                                a["K"], a["dt"], a["act"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), "EDTYPE"), (dict(M=-1), "EINVAL"), (dict(N=0), "EINVAL"), (dict(K=0), "EINVAL"), (dict(act=4), "EINVAL"),
    (dict(act=-1), "EINVAL"), (dict(M=1 << 40), "ERANGE"), (dict(x=None), "EINVAL"), (dict(w=None), "EINVAL"),
    (dict(out=None), "EINVAL"), (dict(ldx=63), "EINVAL"), (dict(ldo=31), "EINVAL"), (dict(ldr=31), "EINVAL"),
    (dict(ldx=1 << 60), "EINVAL"), (dict(ws=WS, wsb=-1), "EINVAL"), (dict(ws=WS + 16, wsb=1024), "EINVAL"),
    (dict(N=(1 << 30) + 1, ldo=1 << 31, ldr=1 << 31), "ERANGE"), (dict(N=1 << 30, K=1 << 30, M=1), "ERANGE"),
    (dict(out=X), "EINVAL"), (dict(out=W + 100), "EINVAL"), (dict(out=BI), "EINVAL"), (dict(out=RE + 2), "EINVAL"),
    (dict(res=OUT, ldr=40), "EINVAL"), (dict(ws=X - 256, wsb=512), "EINVAL"), (dict(ws=OUT - 256, wsb=512), "EINVAL"),
])
def test_linear_refuses(N, kw, code):
    assert _linear(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def test_linear_accepts_no_rows(N):
    assert _linear(N, M=0, x=None, w=None, out=None) == 0
    assert N.lib.attnres_linear_workspace_size(0, 1, 1, 1) >= 0
    assert N.lib.attnres_linear_workspace_size(-1, 1, 1, 1) == N.ATTNRES_EINVAL


def _linear_bwd(N, **kw):
    a = dict(x=X, ldx=64, w=W, bias=BI, g=RE, ldg=32, gx=OUT, gw=OUT + 0x100000, gb=OUT + 0x200000, M=10, N=32, K=64, dt=1,
             act=3, ws=WS, wsb=1 << 24)
    a.update(kw)
    return N.lib.attnres_linear_backward(a["x"], a["ldx"], a["w"], a["bias"], a["g"], a["ldg"], a["gx"], a["gw"], a["gb"],
                                         a["M"], a["N"], a["K"], a["dt"], a["act"], a["ws"], a["wsb"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=-1), "EDTYPE"), (dict(M=-1), "EINVAL"), (dict(x=None), "EINVAL"), (dict(w=None), "EINVAL"), (dict(g=None), "EINVAL"),
    (dict(ldx=1), "EINVAL"), (dict(ldg=31), "EINVAL"), (dict(ws=None), "EINVAL"), (dict(wsb=16), "EINVAL"),
    (dict(ws=WS + 64), "EINVAL"), (dict(gx=X), "EINVAL"), (dict(gx=RE), "EINVAL"), (dict(gw=W), "EINVAL"), (dict(gb=BI), "EINVAL"),
    (dict(gw=OUT), "EINVAL"), (dict(ws=RE - 256), "EINVAL"), (dict(act=9), "EINVAL"),
])
def test_linear_backward_refuses(N, kw, code):
    assert _linear_bwd(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def _qk(N, **kw):
    a = dict(q=X, qs=256, Hq=4, k=W, ks=128, Hk=2, T=5, D=64, dt=1, gq=None, gk=None, eps=1e-5, pos=BI, f=BI + 4096, rot=64,
             inter=0, qo=OUT, qos=256, ko=OUT + 0x100000, kos=128)
    a.update(kw)
    return N.lib.attnres_qk_norm_rope(*[a[n] for n in ("q", "qs", "Hq", "k", "ks", "Hk", "T", "D", "dt", "gq", "gk", "eps", "pos",
                                                       "f", "rot", "inter", "qo", "qos", "ko", "kos")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), "EDTYPE"), (dict(T=-1), "EINVAL"), (dict(D=0), "EINVAL"), (dict(D=1025, qs=9999, ks=9999), "ERANGE"),
    (dict(Hq=0, Hk=0), "EINVAL"), (dict(rot=63), "EINVAL"), (dict(rot=66), "EINVAL"), (dict(rot=-2), "EINVAL"),
    (dict(inter=2), "EINVAL"), (dict(eps=-1.0), "EINVAL"), (dict(eps=float("nan")), "EINVAL"), (dict(qs=255), "EINVAL"),
    (dict(kos=127), "EINVAL"), (dict(q=None), "EINVAL"), (dict(ko=None), "EINVAL"), (dict(pos=None), "EINVAL"),
    (dict(f=None), "EINVAL"), (dict(qo=X + 2), "EINVAL"), (dict(qo=X, qos=512), "EINVAL"), (dict(qo=W), "EINVAL"),
    (dict(ko=OUT + 64), "EINVAL"), (dict(qo=BI), "EINVAL"), (dict(gq=OUT + 8), "EINVAL"),
])
def test_qk_norm_rope_refuses(N, kw, code):
    assert _qk(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def test_qk_norm_rope_backward_refuses(N):
    def call(ws=WS, wsb=1 << 24, gq=OUT, gq_in=RE, dg=BI, T=5):
        return N.lib.attnres_qk_norm_rope_backward(X, 256, 4, None, 0, 0, T, 64, 1, None, None, 1e-5, None, None, 0, 0, gq_in, 256,
                                                   None, 0, gq, 256, None, 0, dg, None, ws, wsb, None)
    assert call(ws=None) == N.ATTNRES_EINVAL
    assert call(gq=X) == N.ATTNRES_EINVAL
    assert call(gq=RE + 16) == N.ATTNRES_EINVAL
    assert call(gq_in=None) == N.ATTNRES_EINVAL
    assert N.lib.attnres_qk_norm_rope_backward_workspace_size(1, 0, 0, 4) == N.ATTNRES_EINVAL


def _att(N, **kw):
    a = dict(q=X, qs=256, k=W, ks=256, v=RE, vs=256, T=9, H=4, Dk=64, Dv=64, dt=1, g=BI, cu=None, n=1, s0=None, s1=None, scale=1.0,
             out=OUT, os=256, ws=WS, wsb=1 << 30)
    a.update(kw)
    return N.lib.attnres_linear_attention(*[a[n] for n in ("q", "qs", "k", "ks", "v", "vs", "T", "H", "Dk", "Dv", "dt", "g", "cu",
                                                           "n", "s0", "s1", "scale", "out", "os", "ws", "wsb")], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), "EDTYPE"), (dict(T=-1), "EINVAL"), (dict(H=0), "EINVAL"), (dict(Dk=0), "EINVAL"), (dict(Dv=257, vs=1 << 20), "ERANGE"),
    (dict(H=70000, qs=1 << 30), "ERANGE"), (dict(n=2), "EINVAL"), (dict(n=0), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(qs=255), "EINVAL"), (dict(os=255), "EINVAL"), (dict(g=None), "EINVAL"), (dict(q=None), "EINVAL"), (dict(out=None), "EINVAL"),
    (dict(T=1 << 33), "ERANGE"), (dict(ws=WS + 64), "EINVAL"), (dict(ws=X), "EINVAL"),
])
def test_linear_attention_refuses(N, kw, code):
    assert _att(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def _step(N, **kw):
    a = dict(q=X, qs=256, k=W, ks=256, v=RE, vs=256, B=9, H=4, Dk=64, Dv=64, dt=1, g=BI, st=WS, ns=9, slots=None, scale=1.0, out=OUT,
             os=256)
    a.update(kw)
    return N.lib.attnres_linear_attention_step(*[a[n] for n in ("q", "qs", "k", "ks", "v", "vs", "B", "H", "Dk", "Dv", "dt", "g", "st",
                                                                "ns", "slots", "scale", "out", "os")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), "EINVAL"), (dict(B=70000), "ERANGE"), (dict(ns=8), "EINVAL"), (dict(ns=-1), "EINVAL"), (dict(st=None), "EINVAL"),
    (dict(out=None), "EINVAL"), (dict(st=X), "EINVAL"), (dict(out=RE), "EINVAL"), (dict(st=OUT), "EINVAL"), (dict(dt=9), "EDTYPE"),
])
def test_step_refuses(N, kw, code):
    assert _step(N, **kw) == getattr(N, "ATTNRES_" + code), N.lib.attnres_last_error()


def test_no_rows_no_slots(N):
    assert _step(N, B=0, q=None, k=None, v=None, out=None, st=None) == 0
    assert _step(N, ns=0, slots=BI + 64) == 0
    assert _att(N, T=0, q=None, k=None, v=None, out=None) == 0


def test_python_checks(N):
    import torch
    import depth_wise_attention_block_gb300 as A
    x = torch.zeros(2, 4)
    with pytest.raises(TypeError, match="CUDA"):
        A.attnres_linear(x, x, x)
    with pytest.raises(ValueError, match="2-d"):
        A.attnres_linear(x[0], x, x)
    with pytest.raises(ValueError, match="activation"):
        A.attnres_linear(x, x, x, activation="relu6")
    with pytest.raises(TypeError, match="dtype"):
        A.attnres_linear(x.half(), x, x)
    with pytest.raises(ValueError, match="heads"):
        A.attnres_qk_norm_rope(x, None, x, None)
    with pytest.raises(ValueError, match="come together"):
        A.attnres_qk_norm_rope(x[None], None, x[None], None, positions=x)
