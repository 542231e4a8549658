"""The fp64 statements of layer norm, gated recurrence and gradient clipping
pinned by closed forms and central differences."""
import math

import numpy as np
import pytest

from oracle import body_oracle as B


def test_layer_norm_closed_forms():
    # two channels: h = +-1 with eps 0, whatever their mean and distance
    y = B.layer_norm(np.array([[3.0, 7.0], [1e6, 1e6 - 1]]), np.array([2.0, 3.0]), np.array([0.5, -0.5]), 0.0)
    assert np.allclose(y, [[-1.5, 2.5], [2.5, -3.5]])
    # a constant row is its bias
    assert np.allclose(B.layer_norm(np.full((1, 5), 4.0), None, np.arange(5.0), 1e-5), [np.arange(5.0)])
    # zero mean and unit variance of the rest
    x = np.random.default_rng(0).normal(size=(3, 40)) * 5 + 2
    y = B.layer_norm(x, None, None, 0.0)
    assert np.allclose(y.mean(1), 0) and np.allclose((y * y).mean(1), 1)


@pytest.mark.parametrize("gain", [False, True])
def test_layer_norm_gradients_are_the_differences(gain):
    r = np.random.default_rng(1)
    x, dy, w, b = r.normal(size=(4, 7)), r.normal(size=(4, 7)), r.normal(size=7), r.normal(size=7)
    if not gain:
        w = None
    dx, dw, db = B.layer_norm_backward(x, w, 1e-3, dy)

    def loss(x, w, b):
        return (B.layer_norm(x, w, b, 1e-3) * dy).sum()
    h = 1e-6
    for _ in range(5):
        u = r.normal(size=x.shape)
        assert math.isclose((loss(x + h * u, w, b) - loss(x - h * u, w, b)) / (2 * h), (dx * u).sum(), rel_tol=1e-6, abs_tol=1e-7)
        u = r.normal(size=7)
        w1 = np.ones(7) if w is None else w
        assert math.isclose((loss(x, w1 + h * u, b) - loss(x, w1 - h * u, b)) / (2 * h), (dw * u).sum(), rel_tol=1e-6, abs_tol=1e-7)
        assert math.isclose((loss(x, w, b + h * u) - loss(x, w, b - h * u)) / (2 * h), (db * u).sum(), rel_tol=1e-6, abs_tol=1e-7)


def test_gated_recurrence_closed_forms():
    assert np.allclose(B.sigmoid(np.array([-800.0, -2.0, 0.0, 2.0, 800.0])), [0, 1 / (1 + math.exp(2)), 0.5, 1 / (1 + math.exp(-2)), 1])
    # a constant gate: a geometric series over a constant input, from any start
    T, f = 12, math.log(3.0)  # a = 3/4
    x, s0 = np.full((T, 2), 5.0), np.array([[1.0, 9.0]])
    out, fin, before = B.gated_recurrence(x, np.full((T, 2), f), None, [0, T], s0)
    want = 5.0 + (s0 - 5.0) * 0.75 ** np.arange(1, T + 1)[:, None]
    assert np.allclose(out, want) and np.allclose(fin, want[-1]) and np.allclose(before[1:], want[:-1]) and np.allclose(before[0], s0)
    # gates wide open and shut: the input, and the state for good
    out, fin, _ = B.gated_recurrence(x, np.array([[-800.0, 800.0]] * T), None, [0, T], s0)
    assert np.allclose(out[:, 0], 5.0) and np.allclose(out[:, 1], 9.0)
    # sequences do not see one another; an empty one hands its state through
    r = np.random.default_rng(2)
    x, f, g, s0 = r.normal(size=(9, 3)), r.normal(size=(9, 3)), r.normal(size=(9, 3)), r.normal(size=(3, 3))
    out, fin, _ = B.gated_recurrence(x, f, g, [1, 5, 5, 8], s0)
    assert np.isnan(out[[0, 8]]).all() and np.allclose(fin[1], s0[1])
    alone, end, _ = B.gated_recurrence(x[5:8], f[5:8], g[5:8], [0, 3], s0[2:])
    assert np.allclose(out[5:8], alone) and np.allclose(fin[2], end[0])
    # the step is the same recurrence
    st, rows = s0.copy(), []
    for t in range(5, 8):
        o, st = B.gated_recurrence_step(x[t:t + 1], f[t:t + 1], g[t:t + 1], st, [2])
        rows.append(o[0])
    assert np.allclose(rows, alone) and np.allclose(st[2], end[0]) and np.allclose(st[:2], s0[:2])
    # rows of one slot follow one another, a row without one is left out
    o, st = B.gated_recurrence_step(x[5:9], f[5:9], g[5:9], s0, [2, 2, 2, -1])
    assert np.allclose(o[:3], alone) and np.isnan(o[3]).all() and np.allclose(st[2], end[0])


@pytest.mark.parametrize("gate", [False, True])
def test_gated_recurrence_gradients_are_the_differences(gate):
    r = np.random.default_rng(3)
    T, C, cu = 8, 3, [0, 3, 3, 8]
    v = dict(x=r.normal(size=(T, C)), f=r.normal(size=(T, C)), g=r.normal(size=(T, C)) if gate else None, s0=r.normal(size=(3, C)))
    dy, ds1 = r.normal(size=(T, C)), r.normal(size=(3, C))
    grads = dict(zip(("x", "f", "g", "s0"), B.gated_recurrence_backward(v["x"], v["f"], v["g"], cu, v["s0"], dy, ds1)))

    def loss(**kw):
        a = {**v, **kw}
        out, fin, _ = B.gated_recurrence(a["x"], a["f"], a["g"], cu, a["s0"])
        return (out * dy).sum() + (fin * ds1).sum()
    h = 1e-6
    for name, val in v.items():
        if val is None:
            assert grads[name] is None
            continue
        for _ in range(4):
            u = r.normal(size=val.shape)
            want = (loss(**{name: val + h * u}) - loss(**{name: val - h * u})) / (2 * h)
            assert math.isclose(want, (grads[name] * u).sum(), rel_tol=1e-6, abs_tol=1e-7), name


def test_grad_clip_closed_forms():
    g = [np.array([3.0]), np.array([[0.0, 4.0]])]
    assert B.grad_clip(g, 10.0)[0] == 5.0 and B.grad_clip(g, 10.0)[1][1][0, 1] == 4.0
    norm, out = B.grad_clip(g, 1.0)
    assert norm == 5.0 and np.allclose(out[0], 0.6) and np.allclose(out[1], [[0, 0.8]])
    assert B.grad_clip([np.array([np.inf, 1.0])], 1.0)[1][0][1] == 1.0
    assert B.grad_clip([np.zeros(4)], 0.0)[0] == 0.0
