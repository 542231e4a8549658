"""Projections whose bf16 rows lie off the 16-byte boundaries: through the copy
to the tensor cores where the workspace is the wrapper's, on the CUDA cores
where the caller's has no room for it.  Bounds as in test_gpu_body_ops.py."""
import pytest
import torch

from oracle import body_oracle as B
from test_gpu_body_ops import E, U, _close, _err, _linear_bound, _randn, _gen, to64

pytestmark = pytest.mark.gpu
DT = torch.bfloat16


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def _off(t, by, pad):
    """The same values in rows that start `by` elements into rows `pad` longer."""
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device="cuda")
    view = wide[:, by:by + t.shape[1]]
    view.copy_(t)
    return view


def _flat_off(t, by):
    """The same values, contiguous, `by` elements behind a boundary."""
    flat = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
    view = flat[by:].view(t.shape)
    view.copy_(t)
    return view


def _inputs(m, n, k, dt=DT, seed=1):
    g = _gen(seed)
    return _randn(g, m, k, dtype=dt), _randn(g, n, k, dtype=dt, scale=k ** -0.5), _randn(g, n, scale=0.3), _randn(g, m, n, dtype=dt)


# x off by one element, an odd row stride, w inside a packed buffer, everything
PLACES = {"x": (1, 8, 0), "stride": (0, 1, 0), "w": (0, 0, 3), "both": (4, 12, 5)}


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("m,n,k", [(1, 264, 512), (64, 1000, 1024), (300, 264, 520), (2100, 2600, 200)])
def test_unaligned_rows_take_the_aligned_path(A, m, n, k, place):
    """A copy to aligned rows and the same kernels: the same bits as aligned
    operands give."""
    by, pad, wby = PLACES[place]
    x, w, b, gy = _inputs(m, n, k)
    xo, wo = (_off(x, by, pad) if pad else x), (_flat_off(w, wby) if wby else w)
    want, got = torch.empty(m, n, dtype=DT, device="cuda"), torch.empty(m, n, dtype=DT, device="cuda")
    err = _err()
    A.attnres_linear(x, w, want, bias=b, activation="silu", dev_err=err)
    A.attnres_linear(xo, wo, got, bias=b, activation="silu", dev_err=err)
    assert torch.equal(want, got)
    for act in ("none", "silu"):
        grads = [[torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")] for _ in range(3)]
        A.attnres_linear_backward(x, w, gy, *grads[0], bias=b, activation=act, dev_err=err)
        A.attnres_linear_backward(xo, wo, gy, *grads[1], bias=b, activation=act, dev_err=err)
        A.attnres_linear_backward(x, w, _off(gy, by, pad) if pad else gy, *grads[2], bias=b, activation=act, dev_err=err)
        for other in grads[1:]:
            assert all(torch.equal(p, q) for p, q in zip(grads[0], other)), act
    assert int(err.item()) == 0


def test_a_workspace_of_the_operands_size_suffices(A):
    """Asked with the operands, the size makes room for their copies; asked by
    sizes alone it is that of aligned ones."""
    m, n, k = 300, 264, 520
    x, w, b, gy = _inputs(m, n, k)
    xo = _off(x, 1, 8)
    assert A.attnres_linear_workspace_size(m, n, k, DT) == A.attnres_linear_workspace_size(m, n, k, DT, x=x, w=w) == 0
    need = A.attnres_linear_workspace_size(m, n, k, DT, x=xo, w=w)
    assert need >= m * k * 2
    want, got = torch.empty(m, n, dtype=DT, device="cuda"), torch.empty(m, n, dtype=DT, device="cuda")
    A.attnres_linear(x, w, want)
    A.attnres_linear(xo, w, got, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(want, got)
    less = A.attnres_linear_backward_workspace_size(m, n, k, DT, "silu")
    need = A.attnres_linear_backward_workspace_size(m, n, k, DT, "silu", x=xo, w=w, grad_out=gy)
    assert need >= less + m * k * 2 and A.attnres_linear_backward_workspace_size(m, n, k, DT, "silu", x=x, w=w, grad_out=gy) == less
    a, c = [torch.empty_like(x), torch.empty_like(w)], [torch.empty_like(x), torch.empty_like(w)]
    A.attnres_linear_backward(x, w, gy, *a, activation="silu")
    A.attnres_linear_backward(xo, w, gy, *c, activation="silu", workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(a, c))


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dt,m,n,k", [(DT, 1, 1, 1), (DT, 3, 70, 8), (DT, 65, 127, 136), (DT, 130, 64, 200), (torch.float32, 65, 127, 131),
                                      (torch.float32, 3, 200, 1000)])
def test_the_cuda_cores_without_a_workspace(A, m, n, k, dt, act):
    """bf16 rows off the boundaries and fp32 above the small products, whose
    copies have no place: the plain kernel, odd edges, fp64 bounds."""
    x, w, b, res = _inputs(m, n, k, dt, 7)
    xo = _off(x, 1, 9)
    wide = torch.full((m, n + 5), 7.0, dtype=dt, device="cuda")
    out = wide[:, 3:3 + n]
    err = _err()
    A.attnres_linear(xo, w, out, bias=b, residual=res, activation=act, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"), dev_err=err)
    want = B.linear(to64(x), to64(w), to64(b), to64(res), act)
    _close(out, want, _linear_bound(to64(x), to64(w), to64(b), to64(res), dt, act, want), "out")
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + n:] == 7).all() and int(err.item()) == 0


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (65, 128, 136), (130, 64, 200), (700, 72, 40)])
def test_the_backward_on_the_cuda_cores(A, m, n, k, act):
    """bf16, a workspace for aligned rows and rows that are not: no room for
    their copy.  (N and K multiples of 8, else the sizes ask for one.)"""
    x, w, b, gy = _inputs(m, n, k, DT, 8)
    xo = _off(x, 1, 9)
    gx, gw, gb = torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")
    ws = torch.empty(A.attnres_linear_backward_workspace_size(m, n, k, DT, act), dtype=torch.uint8, device="cuda")
    err = _err()
    A.attnres_linear_backward(xo, w, gy, gx, gw, gb, bias=b, activation=act, workspace=ws, dev_err=err)
    assert int(err.item()) == 0
    x64, w64, g64, b64 = to64(x), to64(w), to64(gy), to64(b)
    dx, dw, db, dz = B.linear_backward(x64, w64, g64, b64, act)
    import numpy as np
    cz = np.abs(x64) @ np.abs(w64).T + np.abs(b64)
    ez = np.abs(g64) * (0 if act == "none" else 1.2 * (k + 16) * E * cz + 12 * E * 1.13)
    ezr = ez + (0 if act == "none" else U[DT] * np.abs(dz))
    _close(gx, dx, U[DT] * np.abs(dx) + (ezr + (n + 16) * E * np.abs(dz)) @ np.abs(w64), "grad_x")
    _close(gw, dw, U[DT] * np.abs(dw) + (ezr + (m + 16) * E * np.abs(dz)).T @ np.abs(x64), "grad_w")
    _close(gb, db, (ez + (m + 16) * E * np.abs(dz)).sum(0), "grad_bias")
