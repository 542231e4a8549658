"""Plain fp64 statements of a layer body's operators and their gradients:
projection with its epilogue, head norms with rotation, linear attention with
a decay per head.  Written from the formulas, token by token where there is a
recurrence; pinned by tests/test_body_oracle.py (closed forms, central
differences).
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


# ------------------------------------------------------------- projection --

def activation(z, kind):
    if kind == "gelu":
        return z * 0.5 * (1.0 + _erf(z / math.sqrt(2.0)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z / (1.0 + np.exp(-z))
    assert kind == "none"
    return z


def activation_slope(z, kind):
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 0.134145 * z * z)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    assert kind == "none"
    return np.ones_like(z)


def linear(x, w, bias=None, residual=None, act="none"):
    z = x @ w.T + (0.0 if bias is None else bias)
    return activation(z, act) + (0.0 if residual is None else residual)


def linear_backward(x, w, g, bias=None, act="none"):
    """(dx, dw, dbias, dz) for the incoming gradient g."""
    dz = g * activation_slope(x @ w.T + (0.0 if bias is None else bias), act)
    return dz @ w, dz.T @ x, dz.sum(0), dz


# ------------------------------------------------------ norm and rotation --

def rotation_pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def qk_norm_rope(x, gain, positions, inv_freq, interleaved, eps):
    """x [T, H, D]; gain [D] or None; angles positions[t] * inv_freq[i]."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if gain is not None:
        y = y * gain
    a, b = rotation_pairs(2 * len(inv_freq), interleaved)
    ang = positions[:, None, None].astype(np.float64) * inv_freq
    out = y.copy()
    out[..., a] = y[..., a] * np.cos(ang) - y[..., b] * np.sin(ang)
    out[..., b] = y[..., b] * np.cos(ang) + y[..., a] * np.sin(ang)
    return out


def qk_norm_rope_backward(x, gain, positions, inv_freq, interleaved, eps, dout):
    """(dx, dgain)."""
    a, b = rotation_pairs(2 * len(inv_freq), interleaved)
    ang = positions[:, None, None].astype(np.float64) * inv_freq
    dy = dout.copy()
    dy[..., a] = dout[..., a] * np.cos(ang) + dout[..., b] * np.sin(ang)
    dy[..., b] = dout[..., b] * np.cos(ang) - dout[..., a] * np.sin(ang)
    rho = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    hat = x / rho
    n = dy if gain is None else dy * gain
    return (n - hat * (n * hat).mean(-1, keepdims=True)) / rho, (dy * hat).sum((0, 1))


# -------------------------------------------------------- linear attention --

def linear_attention(q, k, v, log_decay, cu, s0, scale):
    """(out, final states) of the recurrence; rows outside every sequence NaN."""
    lam = np.exp(log_decay)[:, None, None]
    n, (T, H, Dk), Dv = len(cu) - 1, q.shape, v.shape[2]
    out = np.full((T, H, Dv), np.nan)
    fin = np.zeros((n, H, Dk, Dv)) if s0 is None else s0.copy()
    for i in range(n):
        for t in range(cu[i], cu[i + 1]):
            fin[i] = lam * fin[i] + k[t][:, :, None] * v[t][:, None, :]
            out[t] = scale * (q[t][:, None, :] @ fin[i])[:, 0]
    return out, fin


def linear_attention_backward(q, k, v, log_decay, cu, s0, scale, do, ds1):
    """(dq, dk, dv, d initial state)."""
    lam = np.exp(log_decay)[:, None, None]
    n, (T, H, Dk), Dv = len(cu) - 1, q.shape, v.shape[2]
    dq, dk, dv = np.full((T, H, Dk), np.nan), np.full((T, H, Dk), np.nan), np.full((T, H, Dv), np.nan)
    ds0 = np.zeros((n, H, Dk, Dv)) if ds1 is None else ds1.copy()
    for i in range(n):
        S = np.zeros((H, Dk, Dv)) if s0 is None else s0[i].copy()
        for t in range(cu[i], cu[i + 1]):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * (S @ do[t][:, :, None])[..., 0]
        for t in range(cu[i + 1] - 1, cu[i] - 1, -1):
            ds0[i] += scale * q[t][:, :, None] * do[t][:, None, :]
            dk[t] = (ds0[i] @ v[t][:, :, None])[..., 0]
            dv[t] = (k[t][:, None, :] @ ds0[i])[:, 0]
            ds0[i] *= lam
    return dq, dk, dv, ds0


def linear_attention_step(q, k, v, log_decay, state, slots, scale):
    """(out, states): rows in order; a row without a slot gives NaN."""
    lam = np.exp(log_decay)[:, None, None]
    state, out = state.copy(), np.full(v.shape, np.nan)
    for b, s in enumerate(slots):
        if 0 <= s < len(state):
            state[s] = lam * state[s] + k[b][:, :, None] * v[b][:, None, :]
            out[b] = scale * (q[b][:, None, :] @ state[s])[:, 0]
    return out, state
