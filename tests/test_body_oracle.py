"""Pins of the layer body's fp64 statements: closed forms, and every gradient
against central differences of its forward."""
import math

import numpy as np
import pytest

from oracle import body_oracle as B

H = 1e-6


def _rng(seed):
    return np.random.default_rng(seed)


def _differences(f, x, g):
    """Gradient of sum(f(x) g) by central differences."""
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        x0 = x[i]
        x[i] = x0 + H
        up = (f() * g).sum()
        x[i] = x0 - H
        dn = (f() * g).sum()
        x[i] = x0
        d[i] = (up - dn) / (2 * H)
    return d


# central differences of step H: truncation of order H^2, rounding of order
# 1e-16 |f| / H with |f| of order 10 here: 1e-8 of the values' size, times 100
TOL = 1e-6


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])
def test_linear_gradients_are_the_differences(act):
    r = _rng(1)
    x, w, b, g = r.normal(size=(3, 5)), r.normal(size=(4, 5)), r.normal(size=4), r.normal(size=(3, 4))
    dx, dw, db, _ = B.linear_backward(x, w, g, b, act)
    for got, var in ((dx, x), (dw, w), (db, b)):
        np.testing.assert_allclose(got, _differences(lambda: B.linear(x, w, b, None, act), var, g), atol=TOL, rtol=TOL)


def test_activations_at_known_points():
    z = np.array([0.0, 1.0, -1.0])
    np.testing.assert_allclose(B.activation(z, "silu"), [0, 1 / (1 + math.exp(-1)), -1 / (1 + math.e)], rtol=1e-14)
    np.testing.assert_allclose(B.activation(z, "gelu"), [0, 0.8413447460685429, -0.15865525393145707], rtol=1e-12)
    assert abs(B.activation(z, "gelu_tanh") - B.activation(z, "gelu")).max() < 2e-3


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 6])
def test_norm_rotation_gradients_are_the_differences(interleaved, rot):
    r = _rng(2)
    x, gain, g = r.normal(size=(3, 2, 6)), r.normal(size=6), r.normal(size=(3, 2, 6))
    pos, f = np.array([0, 5, 1000]), 1.0 / 10.0 ** np.arange(rot // 2)
    dx, dgain = B.qk_norm_rope_backward(x, gain, pos, f, interleaved, 1e-5, g)
    fwd = lambda: B.qk_norm_rope(x, gain, pos, f, interleaved, 1e-5)  # noqa: E731
    np.testing.assert_allclose(dx, _differences(fwd, x, g), atol=TOL, rtol=TOL)
    np.testing.assert_allclose(dgain, _differences(fwd, gain, g), atol=TOL, rtol=TOL)


def test_rotation_keeps_lengths_and_relative_positions():
    r = _rng(3)
    x, f = r.normal(size=(1, 1, 8)), 1.0 / 10.0 ** np.arange(4)
    def at(p, v):
        return B.qk_norm_rope(v, None, np.array([p]), f, False, 0.0)[0, 0]
    assert abs(np.square(at(7, x)).mean() - 1) < 1e-12
    y = r.normal(size=(1, 1, 8))
    assert abs(at(100, x) @ at(93, y) - at(27, x) @ at(20, y)) < 1e-10


def _attention_inputs(seed, T, H_, Dk, Dv, n):
    r = _rng(seed)
    cu = np.concatenate([[0], np.sort(r.integers(0, T + 1, n - 1)), [T]])
    return (r.normal(size=(T, H_, Dk)), r.normal(size=(T, H_, Dk)), r.normal(size=(T, H_, Dv)),
            -r.uniform(0, 1, H_), cu, r.normal(size=(n, H_, Dk, Dv)))


def test_attention_is_the_decayed_triangle():
    q, k, v, g, cu, s0 = _attention_inputs(4, 12, 2, 3, 5, 3)
    out, fin = B.linear_attention(q, k, v, g, cu, s0, 0.7)
    for n in range(3):
        a, b = cu[n], cu[n + 1]
        for h in range(2):
            i = np.arange(b - a)
            D = np.where(i[:, None] >= i[None, :], np.exp(g[h] * (i[:, None] - i[None, :])), 0.0)
            want = (q[a:b, h] @ k[a:b, h].T * D) @ v[a:b, h] + np.exp(g[h] * (i + 1))[:, None] * (q[a:b, h] @ s0[n, h])
            np.testing.assert_allclose(out[a:b, h], 0.7 * want, atol=1e-12)
            w = np.exp(g[h] * (b - a - 1 - i))
            np.testing.assert_allclose(fin[n, h], np.exp(g[h] * (b - a)) * s0[n, h] + (k[a:b, h] * w[:, None]).T @ v[a:b, h],
                                       atol=1e-12)


def test_attention_gradients_are_the_differences():
    q, k, v, g, cu, s0 = _attention_inputs(5, 7, 2, 3, 2, 2)
    r = _rng(6)
    do, ds1 = r.normal(size=v.shape), r.normal(size=s0.shape)
    got = B.linear_attention_backward(q, k, v, g, cu, s0, 0.5, do, ds1)

    def fwd():
        out, fin = B.linear_attention(q, k, v, g, cu, s0, 0.5)
        return np.concatenate([(out * do).ravel(), (fin * ds1).ravel()])
    for have, var in zip(got, (q, k, v, s0)):
        np.testing.assert_allclose(have, _differences(fwd, var, 1.0), atol=TOL, rtol=TOL)


def test_steps_are_the_prompt_token_by_token():
    q, k, v, g, _, s0 = _attention_inputs(7, 6, 2, 3, 4, 1)
    out, fin = B.linear_attention(q, k, v, g, [0, 6], s0, 0.3)
    got, st = B.linear_attention_step(q, k, v, g, s0, [0] * 6, 0.3)
    np.testing.assert_allclose(got, out, atol=1e-13)
    np.testing.assert_allclose(st, fin, atol=1e-13)
    got, st = B.linear_attention_step(q, k, v, g, s0, [1, -1, 5, 1, 1, 1], 0.3)
    assert np.isnan(got).all() and (st == s0).all()
