"""attnres_layer_norm and its backward on the GPU against their fp64 statements.

Tolerances, derived from the arithmetic before any run.  u is half a rounding
step of the stored type (bf16 2^-8, fp32 2^-24), e = 2^-23 bounds one fp32
operation.  A sum over a row of d channels runs through at most d / 128 + 48
additions on any path (a thread's own channels, a warp, the warps in order), so
it is off by at most s = (d / 128 + 48) 2^-24 of the sum of absolute values.
The mean is held as two numbers: x - mean is off by 2^-24 of itself and by s
times the mean |x - mean| (at most the row's spread), however far the mean is
from zero.  With h = (x - mean) / sigma and r = 1 / sigma (off by s + 2^-21 of
itself):
  h      |err| <= eh = (s + 2^-21) |h| + 2 s
  out    |gain| eh + e (|gain h| + |bias|) + u |out|
  dx     r ((s + 2^-21) (|n| + (1 + |h|) (2 mean|n| + 4 mean|n h|)) + eh mean|n h|) + (s + 2^-20 + u) |dx|
  dgain  sum |dy| eh, and (T / 128 + 64) e of sum |dy h|
  dbias  (T / 128 + 64) e of sum |dy|
"""
import numpy as np
import pytest
import torch

from oracle import body_oracle as B

pytestmark = pytest.mark.gpu
E = 2.0 ** -23
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def to64(t):
    return t.detach().double().cpu().numpy()


def _randn(seed, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def _close(got, want, bound, what):
    got = to64(got)
    assert np.isfinite(got).all(), what
    err = np.abs(got - want)
    worst = (err / np.maximum(bound, 1e-300)).max() if err.size else 0.0
    assert (err <= bound).all(), f"{what}: worst {worst:.3g} x bound"


def _parts(x, eps):
    z = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
    s = (x.shape[1] / 128 + 48) * 2.0 ** -24
    h = z * r
    return h, r, s, (s + 2.0 ** -21) * np.abs(h) + 2 * s


def _check_forward(x, gain, bias, out, eps, dt, what):
    x, gain, bias = to64(x), None if gain is None else to64(gain), None if bias is None else to64(bias)
    h, _, _, eh = _parts(x, eps)
    w = 1.0 if gain is None else np.abs(gain)
    want = B.layer_norm(x, gain, bias, eps)
    _close(out, want, w * eh + E * (w * np.abs(h) + (0 if bias is None else np.abs(bias))) + U[dt] * np.abs(want), what)


def _check_backward(x, gain, dy, gx, gg, gb, eps, dt, what):
    x, dy, gain = to64(x), to64(dy), None if gain is None else to64(gain)
    dx, dg, db = B.layer_norm_backward(x, gain, eps, dy)
    h, r, s, eh = _parts(x, eps)
    n = np.abs(dy if gain is None else dy * gain)
    mn, mnh = n.mean(-1, keepdims=True), (n * np.abs(h)).mean(-1, keepdims=True)
    err = r * ((s + 2.0 ** -21) * (n + (1 + np.abs(h)) * (2 * mn + 4 * mnh)) + eh * mnh)
    if gx is not None:
        _close(gx, dx, err + (s + 2.0 ** -20 + U[dt]) * np.abs(dx), (what, "grad_x"))
    depth = (x.shape[0] / 128 + 64) * E
    if gg is not None:
        _close(gg, dg, (np.abs(dy) * (eh + depth * np.abs(h))).sum(0), (what, "grad_gain"))
    if gb is not None:
        _close(gb, db, depth * np.abs(dy).sum(0), (what, "grad_bias"))


# widths of one element, of less than a vector and a warp, odd, whole vectors
# for either type, more than one CTA holds at once
SIZES = [(1, 1), (3, 2), (5, 7), (9, 8), (17, 31), (64, 64), (33, 100), (7, 129), (130, 256), (5, 500), (300, 517), (40, 1003), (11, 1024),
         (2, 2056), (65, 4100), (6, 7168), (3, 8193), (2, 12288), (5, 16384), (2, 20000), (1, 40001), (700, 48)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,d", SIZES)
def test_layer_norm(A, T, d, dt):
    eps = 1e-5
    for seed, (gain, bias, wide, shift) in enumerate([(True, True, 0, 0.0), (False, False, 0, 3.0), (True, False, 16, -30.0),
                                                      (False, True, 5, 0.5)]):
        # rows of a wider buffer: on the 16-byte boundaries or off them
        base = _randn(seed, T, d + 2 * wide, dtype=dt, scale=2.0, shift=shift)
        x = base[:, wide:wide + d]
        w = _randn(seed + 10, d, shift=1.0, scale=0.3) if gain else None
        b = _randn(seed + 20, d) if bias else None
        buf = torch.full((T, d + 2 * wide), 7.0, dtype=dt, device="cuda")
        out = buf[:, wide:wide + d]
        A.attnres_layer_norm(x, out, gain=w, bias=b, eps=eps)
        _check_forward(x, w, b, out, eps, dt, (gain, bias, wide))
        assert (buf[:, :wide] == 7).all() and (buf[:, wide + d:] == 7).all()
        dy = _randn(seed + 30, T, d + 2 * wide, dtype=dt)[:, wide:wide + d]
        gx, gg, gb = buf[:, wide:wide + d], torch.full((d,), float("nan"), device="cuda"), torch.full((d,), float("nan"), device="cuda")
        A.attnres_layer_norm_backward(x, dy, gx, gain=w, grad_gain=gg, grad_bias=gb, eps=eps)
        _check_backward(x, w, dy, gx, gg, gb, eps, dt, (gain, bias, wide))
        assert (buf[:, :wide] == 7).all() and (buf[:, wide + d:] == 7).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,d", [(2000, 64), (1500, 1003), (1000, 7168), (5000, 520)])
def test_many_rows(A, T, d, dt):
    """More rows than CTAs run at once: several to each, in both directions."""
    x, dy, w, b = _randn(1, T, d, dtype=dt), _randn(2, T, d, dtype=dt), _randn(3, d), _randn(4, d)
    out, gx, gg, gb = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    A.attnres_layer_norm(x, out, gain=w, bias=b, eps=1e-5)
    _check_forward(x, w, b, out, 1e-5, dt, "forward")
    A.attnres_layer_norm_backward(x, dy, gx, gain=w, grad_gain=gg, grad_bias=gb, eps=1e-5)
    _check_backward(x, w, dy, gx, gg, gb, 1e-5, dt, "backward")


@pytest.mark.parametrize("d", [300, 1024, 7168, 30000])
def test_a_mean_far_from_zero_keeps_the_digits(A, d):
    """fp32 rows around 3e4 with a spread of 1, on the same bars."""
    x, dy = _randn(1, 9, d, shift=3e4), _randn(2, 9, d)
    out, gx, gg, gb = torch.empty_like(x), torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    A.attnres_layer_norm(x, out, eps=1e-5)
    _check_forward(x, None, None, out, 1e-5, torch.float32, "forward")
    A.attnres_layer_norm_backward(x, dy, gx, grad_gain=gg, grad_bias=gb, eps=1e-5)
    _check_backward(x, None, dy, gx, gg, gb, 1e-5, torch.float32, "backward")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("d", [24, 333, 7168])
def test_in_place_and_single_gradients(A, d, dt):
    x, dy, w, b = _randn(1, 200, d, dtype=dt), _randn(2, 200, d, dtype=dt), _randn(3, d), _randn(4, d)
    out, gx, gg, gb = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    A.attnres_layer_norm(x, out, gain=w, bias=b)
    y = x.clone()
    A.attnres_layer_norm(y, y, gain=w, bias=b)
    assert torch.equal(y, out)
    A.attnres_layer_norm_backward(x, dy, gx, gain=w, grad_gain=gg, grad_bias=gb)
    g = dy.clone()
    A.attnres_layer_norm_backward(x, g, g, gain=w)
    assert torch.equal(g, gx)
    for kw in (dict(grad_gain=torch.empty_like(w)), dict(grad_bias=torch.empty_like(w))):
        A.attnres_layer_norm_backward(x, dy, None, gain=w, **kw)
        got, want = (kw["grad_gain"], gg) if "grad_gain" in kw else (kw["grad_bias"], gb)
        assert torch.equal(got, want)
    # the same bits again
    gg2 = torch.empty_like(w)
    A.attnres_layer_norm_backward(x, dy, gx, gain=w, grad_gain=gg2)
    assert torch.equal(gg, gg2)


@pytest.mark.parametrize("d", [40, 1003, 7168])
def test_rows_do_not_see_one_another(A, d):
    """Infinities and NaN of a row stay in it; a constant row is its bias; no
    rows leave zero gradients."""
    x, dy = _randn(1, 6, d), _randn(2, 6, d)
    b = _randn(3, d)
    out, gx = torch.empty_like(x), torch.empty_like(x)
    A.attnres_layer_norm(x, out, bias=b)
    A.attnres_layer_norm_backward(x, dy, gx)
    want, want_g = out.clone(), gx.clone()
    x[1, d // 2], x[3, 0], x[4] = float("inf"), float("nan"), 2.5
    A.attnres_layer_norm(x, out, bias=b)
    A.attnres_layer_norm_backward(x, dy, gx)
    rest = [0, 2, 5]
    assert torch.equal(out[rest], want[rest]) and torch.equal(gx[rest], want_g[rest])
    assert torch.isnan(out[[1, 3]]).all() and torch.allclose(out[4], b, atol=1e-3)
    gg, gb = torch.ones(d, device="cuda"), torch.ones(d, device="cuda")
    A.attnres_layer_norm_backward(x[:0], dy[:0], gx[:0], grad_gain=gg, grad_bias=gb)
    assert not gg.any() and not gb.any()
    A.attnres_layer_norm(x[:0], out[:0])


def test_streams_and_graphs(A):
    x, dy, w = _randn(1, 3000, 1024, dtype=torch.bfloat16), _randn(2, 3000, 1024, dtype=torch.bfloat16), _randn(3, 1024)
    out, gx, gg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    A.attnres_layer_norm(x, out, gain=w, stream=side)
    A.attnres_layer_norm_backward(x, dy, gx, gain=w, grad_gain=gg, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in (out, gx, gg)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.attnres_layer_norm(x, out, gain=w)
        A.attnres_layer_norm_backward(x, dy, gx, gain=w, grad_gain=gg)
    for t in (out, gx, gg):
        t.zero_()
    for _ in range(2):
        graph.replay()
    for t, v in zip((out, gx, gg), want):
        assert torch.equal(t, v)


@pytest.mark.parametrize("dt", DTYPES)
def test_autograd(A, dt):
    """Any leading dimensions, rows in any order in memory, every subset of gradients."""
    from depth_wise_attention_block_gb300 import autograd as F
    x = _randn(1, 4, 96, 5, dtype=dt).transpose(1, 2)
    w, b = _randn(2, 96), _randn(3, 96)
    dy = _randn(4, 4, 5, 96, dtype=dt)
    for need in [(True, True, True), (True, False, False), (False, True, False), (False, False, True)]:
        leaves = [t.detach().clone().requires_grad_(n) for t, n in zip((x, w, b), need)]
        y = F.layer_norm(*leaves)
        assert y.shape == x.shape
        y.backward(dy)
        for t, n in zip(leaves, need):
            assert (t.grad is not None) == n
        gx, gg, gb = (t.grad for t in leaves)
        flat = lambda t: None if t is None else t.reshape(-1, 96)  # noqa: E731
        _check_backward(flat(x), w, flat(dy), flat(gx), gg, gb, 1e-5, dt, need)
    y = F.layer_norm(x)
    _check_forward(x.reshape(-1, 96), None, None, y.reshape(-1, 96), 1e-5, dt, "no vectors")
