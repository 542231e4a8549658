"""attnres_grad_clip on the GPU against its fp64 statement.

Tolerances, derived before any run: a thread adds at most 34 squares in fp32
between two additions in fp64, so the sum of squares is off by 35 2^-24 of
itself and the norm by half of that and its own rounding: n = 19 2^-24.  A
clipped value: n and three fp32 roundings, then its own (u: bf16 2^-8, fp32
2^-24) and fp32's smallest number."""
import math

import numpy as np
import pytest
import torch

from oracle import body_oracle as B

pytestmark = pytest.mark.gpu
N_ERR = 19 * 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
MIXES = [(torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)]


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def to64(t):
    return t.detach().double().cpu().numpy()


def _grads(sizes, dts, seed=0, scale=1.0, shift=0):
    """Tensors of `sizes`, views `shift` elements into buffers of their own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + shift, generator=g, device="cuda") * (scale * 10.0 ** -(i % 4))
        out.append(t.to(dts[i % len(dts)])[shift:])
    return out


def _check(A, grads, max_norm, outs=None):
    ins = [to64(t) for t in grads]
    want_norm, want = B.grad_clip(ins, max_norm)
    norm = torch.full((1,), -1.0, device="cuda")
    res = grads if outs is None else outs
    before = [t.clone() for t in grads]
    A.attnres_grad_clip(grads, max_norm, norm, outs=outs)
    torch.cuda.synchronize()
    if math.isfinite(want_norm) and want_norm < 3.4e38:
        assert abs(float(norm) - want_norm) <= N_ERR * want_norm + 2.0 ** -149
    for t, w in zip(res, want):
        assert (np.abs(to64(t) - w) <= (U[t.dtype] + N_ERR + 3 * 2.0 ** -24) * np.abs(w) + 2.0 ** -133).all()
    if outs is not None:
        for t, b in zip(grads, before):
            assert torch.equal(t, b)
    if want_norm <= max_norm:
        for t, b in zip(res, before):
            assert torch.equal(t, b)
    return float(norm)


# one element; less than a vector; tails; more tensors than one launch takes;
# chunks that end inside a tensor
LISTS = [[1], [3, 5], [7, 0, 8, 1, 9], [8191, 8192, 8193, 16], [1] * 70, [5 + i % 13 for i in range(1000)], [100001, 3, 70000, 1 << 20],
         [4096 * 33 + 17] * 9]


@pytest.mark.parametrize("dts", MIXES)
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_grad_clip(A, sizes, dts):
    for shift in (0, 1, 8):
        grads = _grads(sizes, dts, seed=shift, shift=shift)
        total = math.sqrt(sum(float((to64(t) ** 2).sum()) for t in grads))
        outs = [torch.full_like(t, 5.0) for t in grads]  # (with a shift of 1: otherwise on the 16-byte boundaries)
        _check(A, grads, 0.25 * total, outs)
        _check(A, grads, 4.0 * total, outs)
        _check(A, grads, 4.0 * total)
        _check(A, grads, 0.25 * total)


def test_neighbours_are_left_alone(A):
    for dt in U:
        buf = torch.ones(5000, dtype=dt, device="cuda")
        parts = [buf[i * 100 + 3:i * 100 + 3 + 50 + i] for i in range(40)]
        keep = torch.ones(5000, dtype=torch.bool, device="cuda")
        for i in range(40):
            keep[i * 100 + 3:i * 100 + 3 + 50 + i] = False
        norm = torch.empty(1, device="cuda")
        A.attnres_grad_clip(parts, 0.5, norm)
        assert (buf[keep] == 1).all() and (buf[~keep] < 0.1).all()


def test_the_norm_alone(A):
    grads = _grads([10, 5000, 77], (torch.float32, torch.bfloat16))
    before = [t.clone() for t in grads]
    assert _check(A, grads, float("inf")) > 0
    for t, b in zip(grads, before):
        assert torch.equal(t, b)
    norm = torch.ones(1, device="cuda")
    A.attnres_grad_clip([], 1.0, norm)
    assert float(norm) == 0.0
    A.attnres_grad_clip([torch.empty(0, device="cuda")], float("inf"), norm.fill_(1))
    assert float(norm) == 0.0


@pytest.mark.parametrize("scale", [1e-37, 1e-30, 1e-22, 1e15, 1e25, 1e34])
def test_squares_beyond_fp32(A, scale):
    """The norm where the squares leave fp32 at either end."""
    for dts in MIXES[:2]:
        grads = _grads([3000, 9, 70001], dts, scale=scale)
        _check(A, grads, 1e-3 * scale, [torch.empty_like(t) for t in grads])
        _check(A, [torch.zeros_like(grads[0]), *grads], 0.1 * scale)


def test_edges_of_the_bound(A):
    z = torch.zeros(100, device="cuda")
    assert _check(A, [z], 0.0) == 0.0 and not z.any()
    g = _grads([100], (torch.float32,))
    _check(A, g, 0.0)
    assert not g[0].any()
    # a norm equal to the bound is not above it
    g = [torch.tensor([3.0, 4.0], device="cuda")]
    assert _check(A, g, 5.0) == 5.0 and g[0].tolist() == [3.0, 4.0]


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), float("-inf")])
def test_a_norm_that_is_not_finite_scales_nothing(A, bad):
    for dt in U:
        grads = _grads([70, 9000], (dt,))
        grads[1][4321] = bad
        before = [t.clone() for t in grads]
        outs = [torch.zeros_like(t) for t in grads]
        norm = torch.zeros(1, device="cuda")
        A.attnres_grad_clip(grads, 1e-3, norm, outs=outs)
        assert not math.isfinite(float(norm))
        for t, o, b in zip(grads, outs, before):
            assert torch.equal(o.nan_to_num(7, 8, 9), b.nan_to_num(7, 8, 9)) and torch.equal(t.nan_to_num(7, 8, 9), b.nan_to_num(7, 8, 9))


def test_streams_graphs_and_the_same_bits(A):
    src = _grads([50000, 3, 70001], (torch.bfloat16, torch.float32))
    grads, norm = [t.clone() for t in src], torch.empty(1, device="cuda")
    ws = torch.empty(A.attnres_grad_clip_workspace_size(), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    A.attnres_grad_clip(grads, 0.5, norm, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want, want_norm = [t.clone() for t in grads], norm.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.attnres_grad_clip(grads, 0.5, norm, workspace=ws)
    for _ in range(2):
        for t, s in zip(grads, src):
            t.copy_(s)
        ws.fill_(255)  # what it held before does not matter
        graph.replay()
        for t, v in zip(grads, want):
            assert torch.equal(t, v)
        assert torch.equal(norm, want_norm)


def test_refusals(A):
    g = _grads([10, 20], (torch.float32,))
    norm = torch.empty(1, device="cuda")
    with pytest.raises(A.AttnresError, match="overlaps"):
        A.attnres_grad_clip([g[0], g[0]], 1.0, norm)
    with pytest.raises(ValueError, match="contiguous"):
        A.attnres_grad_clip([torch.zeros(4, 6, device="cuda")[:, :3]], 1.0, norm)
    with pytest.raises(TypeError, match="dtype"):
        A.attnres_grad_clip([g[0].half()], 1.0, norm)
    with pytest.raises(ValueError, match="outs"):
        A.attnres_grad_clip(g, 1.0, norm, outs=g[:1])
    with pytest.raises(ValueError, match="elements"):
        A.attnres_grad_clip(g, 1.0, norm, outs=[g[1], g[0]])
    with pytest.raises(TypeError):
        A.attnres_grad_clip(g, 1.0, norm, outs=[t.bfloat16() for t in g])
    with pytest.raises(ValueError, match="max_norm"):
        A.attnres_grad_clip(g, float("nan"), norm)
    with pytest.raises(A.AttnresError, match="workspace"):
        A.attnres_grad_clip(g, 1.0, norm, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_clip_grad_norm_of_leaves(A):
    from depth_wise_attention_block_gb300 import autograd as F
    a, b, c = (torch.zeros(n, device="cuda", requires_grad=True) for n in (6, 3, 5))
    a.grad, b.grad = torch.full((6,), 2.0, device="cuda"), torch.full((3,), -1.0, device="cuda")
    norm = F.clip_grad_norm([a, b, c, a], 1.0)  # a leaf without a gradient, one named twice
    want = math.sqrt(27.0)
    assert abs(float(norm) - want) <= N_ERR * want
    assert np.allclose(to64(a.grad), 2 / want, rtol=1e-5) and np.allclose(to64(b.grad), -1 / want, rtol=1e-5) and c.grad is None
    m = torch.zeros(4, 6, device="cuda", requires_grad=True)
    m.grad = torch.ones(6, 4, device="cuda").t()
    assert abs(float(F.clip_grad_norm(m, float("inf"))) - math.sqrt(24.0)) < 1e-5
