"""Which gradients attnres_linear_attention_backward takes as NULL (checked on
the host, before any launch; the pointers are never dereferenced)."""
import pytest

from test_body_refusals import BI, N, OUT, RE, W, WS, X  # noqa: F401


def _call(N, **kw):
    a = dict(go=X + 0x4000000, dq=OUT, dk=OUT + 0x400000, dv=OUT + 0x800000, ds0=None, T=9)
    a.update(kw)
    return N.lib.attnres_linear_attention_backward(X, 256, W, 256, RE, 256, a["T"], 4, 64, 64, 1, BI, None, 1, None, 1.0, a["go"], 256,
                                                   None, a["dq"], a["dk"], a["dv"], a["ds0"], WS, 1 << 30, None, None)


@pytest.mark.parametrize("kw", [dict(go=None), dict(dv=None, ds0=OUT + 0xC00000), dict(dq=None, dk=None, dv=None, ds0=OUT + 0xC00000),
                                dict(dq=X), dict(dk=OUT), dict(dq=None, dk=None, dv=RE), dict(ds0=OUT)])
def test_refused(N, kw):  # noqa: F811
    assert _call(N, **kw) == N.ATTNRES_EINVAL, N.lib.attnres_last_error()


def test_nothing_asked_for(N):  # noqa: F811
    assert _call(N, dq=None, dk=None, dv=None, go=None) == 0


@pytest.mark.parametrize("M", [(1 << 31) - 1, (1 << 31) - 64])
def test_rows_whose_last_step_leaves_an_int(N, M):  # noqa: F811
    """grad_w contracts over the rows 16 at a time, in 32 bits."""
    ws = 1 << 50
    assert N.lib.attnres_linear_backward(X, 8, W, None, 1 << 45, 8, None, OUT, None, M, 8, 8, 1, 0, 1 << 46, ws, None,
                                         None) == N.ATTNRES_ERANGE
    assert N.lib.attnres_linear_backward_workspace_size(M, 8, 8, 1, 0) == N.ATTNRES_ERANGE
    assert N.lib.attnres_linear_workspace_size(M, 8, 8, 1) == N.ATTNRES_ERANGE
    assert N.lib.attnres_linear_workspace_size((1 << 31) - 65, 8, 8, 1) == 0
