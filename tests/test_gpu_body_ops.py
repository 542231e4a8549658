"""The operators of a layer body on the GPU against their fp64 statements.

Tolerances, all derived from the arithmetic before any run.  u is half a
rounding step of the stored type (bf16 2^-8, fp32 2^-24), e = 2^-23 bounds one
fp32 operation (or one truncated step of a tensor core's accumulator), and
`cond` is the same sum over absolute values:
  a sum of K products        |err| <= (K + 16) e cond
  a stored value             + u |value|
  an operand rounded to bf16 before a product: + 2^-8 of that product's cond
  fp32 underflow: a decay's power below 2^-149 is 0, which loses its factor,
                  a sum of products of values of order 1 (below 2^20 for every
                  size here), times less than 2^-149: + 2^-129
"""
import math

import numpy as np
import pytest
import torch

from oracle import body_oracle as B

pytestmark = pytest.mark.gpu
E = 2.0 ** -23
UNDERFLOW = 2.0 ** -129
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def to64(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _close(got, want, bound, what):
    err = np.abs(to64(got) - want)
    assert np.isfinite(to64(got)).all(), what
    worst = (err / np.maximum(bound, UNDERFLOW)).max() if err.size else 0.0
    assert (err <= bound + UNDERFLOW).all(), f"{what}: worst {worst:.3g} x bound"


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ linear --

LINEAR = [(1, 1, 1), (1, 16, 8), (3, 5, 7), (16, 128, 64), (17, 130, 72), (64, 512, 1024), (65, 127, 129), (128, 256, 64),
          (129, 257, 200), (300, 264, 520), (257, 1000, 96), (513, 384, 1600),
          (1, 700, 1100), (40, 1030, 333), (128, 260, 901),
          (64, 12100, 72), (200, 9000, 136), (70, 72, 9000)]  # tiles as wide as make the waves even


def _linear_inputs(m, n, k, dt, seed, strided=False):
    g = _gen(seed)
    if strided:  # slices of wider buffers
        x = _randn(g, m, k + 24, dtype=dt)[:, 8:8 + k]
        res = _randn(g, m, 2 * n + 8, dtype=dt)[:, n:2 * n]
    else:
        x, res = _randn(g, m, k, dtype=dt), _randn(g, m, n, dtype=dt)
    return x, _randn(g, n, k, dtype=dt, scale=k ** -0.5), _randn(g, n, scale=0.3), res


def _linear_bound(x, w, b, res, dt, act, want):
    """The value's own rounding, and the sum's error through a slope of at
    most 1.13 (the largest of the activations'), plus 8 fp32 operations on
    the activation's value and the residual."""
    cond = np.abs(x) @ np.abs(w).T + (0 if b is None else np.abs(b))
    k = x.shape[1]
    big = np.abs(want) + cond + (0 if res is None else np.abs(res))
    return U[dt] * np.abs(want) + 1.13 * (k + 16) * E * cond + 8 * E * big


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear(A, m, n, k, dt):
    for i, (act, bias, resid, strided) in enumerate([("none", False, False, False), ("silu", True, True, True),
                                                     ("gelu", True, False, False), ("gelu_tanh", False, True, False)]):
        x, w, b, res = _linear_inputs(m, n, k, dt, 10 * i + 1, strided)
        b, res = b if bias else None, res if resid else None
        wide = torch.full((m, n + 16), 7.0, dtype=dt, device="cuda")
        out = wide[:, 8:8 + n] if strided else torch.full((m, n), float("nan"), dtype=dt, device="cuda")
        err = _err()
        A.attnres_linear(x, w, out, bias=b, residual=res, activation=act, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        x64, w64 = to64(x), to64(w)
        b64, r64 = None if b is None else to64(b), None if res is None else to64(res)
        want = B.linear(x64, w64, b64, r64, act)
        _close(out, want, _linear_bound(x64, w64, b64, r64, dt, act, want), (act, strided))
        if strided:  # nothing beside the slice was written
            assert (wide[:, :8] == 7).all() and (wide[:, 8 + n:] == 7).all()


@pytest.mark.parametrize("dt", DTYPES)
def test_linear_adds_in_place_and_without_workspace(A, dt):
    x, w, b, res = _linear_inputs(33, 48, 40, dt, 5)
    want = torch.empty_like(res)
    A.attnres_linear(x, w, want, bias=b, residual=res)
    out = res.clone()
    A.attnres_linear(x, w, out, bias=b, residual=out, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    ref = B.linear(to64(x), to64(w), to64(b), to64(res))
    _close(out, ref, _linear_bound(to64(x), to64(w), to64(b), to64(res), dt, "none", ref), "in place")
    _close(want, ref, _linear_bound(to64(x), to64(w), to64(b), to64(res), dt, "none", ref), "apart")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear_backward(A, m, n, k, dt):
    for i, (act, bias, strided) in enumerate([("none", False, False), ("silu", True, True), ("gelu", True, False),
                                              ("gelu_tanh", False, False)]):
        x, w, b, gy = _linear_inputs(m, n, k, dt, 10 * i + 2, strided)
        b = b if bias else None
        gx, gw = torch.empty(m, k, dtype=dt, device="cuda"), torch.empty(n, k, dtype=dt, device="cuda")
        gb = torch.empty(n, device="cuda")
        err = _err()
        A.attnres_linear_backward(x, w, gy, gx, gw, gb, bias=b, activation=act, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        x64, w64, g64, b64 = to64(x), to64(w), to64(gy), None if b is None else to64(b)
        dx, dw, db, dz = B.linear_backward(x64, w64, g64, b64, act)
        # dz: z's error through the slope's own slope (at most 1.2), 12 fp32 operations, then its rounding
        cz = np.abs(x64) @ np.abs(w64).T + (0 if b is None else np.abs(b64))
        ez = np.abs(g64) * (0 if act == "none" else 1.2 * (k + 16) * E * cz + 12 * E * 1.13)
        ezr = ez + (0 if act == "none" else U[dt] * np.abs(dz))
        _close(gx, dx, U[dt] * np.abs(dx) + (ezr + (n + 16) * E * np.abs(dz)) @ np.abs(w64), (act, "grad_x"))
        _close(gw, dw, U[dt] * np.abs(dw) + (ezr + (m + 16) * E * np.abs(dz)).T @ np.abs(x64), (act, "grad_w"))
        _close(gb, db, (ez + (m + 16) * E * np.abs(dz)).sum(0), (act, "grad_bias"))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k,act", [(2100, 2600, 200, "silu"), (4000, 5000, 328, "none"), (2049, 4097, 520, "gelu"),
                                       (1030, 9000, 136, "gelu_tanh")])
def test_linear_many_tiles(A, m, n, k, act, dt):
    """Sizes of several waves of tiles, forward and gradients, with odd edges;
    the fp64 statement evaluated by torch on the GPU, for its speed."""
    x, w, b, res = _linear_inputs(m, n, k, dt, 31)
    out, gx, gw, gb = torch.empty_like(res), torch.empty_like(x), torch.empty_like(w), torch.empty(n, device="cuda")
    err = _err()
    A.attnres_linear(x, w, out, bias=b, residual=res, activation=act, dev_err=err)
    A.attnres_linear_backward(x, w, res, gx, gw, gb, bias=b, activation=act, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    X, Wt, R = x.double(), w.double(), res.double()
    z = (X @ Wt.T + b.double()).cpu().numpy()
    want = torch.from_numpy(B.activation(z, act)).cuda() + R
    cz = X.abs() @ Wt.abs().T + b.double().abs()
    u = U[dt]

    def close(got, ref, bound, what):
        e = (got.double() - ref).abs()
        assert torch.isfinite(got).all() and (e <= bound + UNDERFLOW).all(), f"{what}: worst {(e / (bound + UNDERFLOW)).max():.3g} x bound"
    close(out, want, u * want.abs() + 1.13 * (k + 16) * E * cz + 8 * E * (want.abs() + cz + R.abs()), "out")
    dz = R * torch.from_numpy(B.activation_slope(z, act)).cuda()
    ez = R.abs() * (0 if act == "none" else 1) * (1.2 * (k + 16) * E * cz + 12 * E * 1.13)
    ezr = ez + (0 if act == "none" else u) * dz.abs()
    dx, dw = dz @ Wt, dz.T @ X
    close(gx, dx, u * dx.abs() + (ezr + (n + 16) * E * dz.abs()) @ Wt.abs(), "grad_x")
    close(gw, dw, u * dw.abs() + (ezr + (m + 16) * E * dz.abs()).T @ X.abs(), "grad_w")
    close(gb, dz.sum(0), (ez + (m + 16) * E * dz.abs()).sum(0), "grad_bias")


def test_linear_backward_parts_and_empty(A):
    x, w, b, gy = _linear_inputs(70, 40, 24, torch.bfloat16, 3)
    full = [torch.empty_like(x), torch.empty_like(w), torch.empty(40, device="cuda")]
    A.attnres_linear_backward(x, w, gy, *full, bias=b, activation="silu")
    for i in range(3):  # each gradient on its own: the same bits
        part = [None] * 3
        part[i] = torch.empty_like(full[i])
        A.attnres_linear_backward(x, w, gy, *part, bias=b, activation="silu")
        assert torch.equal(part[i], full[i])
    A.attnres_linear_backward(x[:0], w, gy[:0], full[0][:0], full[1], full[2], bias=b, activation="silu")
    assert not full[1].any() and not full[2].any()
    A.attnres_linear(x[:0], w, gy[:0])


# ------------------------------------------------------------ qk norm rope --

QK = [  # T, Hq, Hk, D, rot
    (1, 1, 1, 64, 64), (5, 3, 1, 128, 128), (64, 56, 8, 128, 128), (33, 4, 2, 96, 64), (17, 2, 2, 96, 96), (9, 2, 1, 80, 0),
    (7, 3, 2, 37, 12), (3, 2, 1, 1, 0), (11, 2, 1, 18, 18), (6, 1, 2, 256, 128), (4, 2, 1, 512, 512), (3, 1, 1, 1000, 10),
    (700, 20, 4, 64, 32), (300, 30, 30, 192, 192),
]


def _qk_inputs(T, Hq, Hk, D, rot, dt, seed, far=0):
    g = _gen(seed)
    rows = _randn(g, T, (Hq + 2 * Hk) * D, dtype=dt, scale=3.0)
    q, k = rows[:, :Hq * D].unflatten(1, (Hq, D)), rows[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    gains = [1 + _randn(g, D, scale=0.3) for _ in range(2)]
    pos = far + torch.randint(0, 5000, (T,), generator=g, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))).float()
    return q, k, gains, pos, freq


def _pair_abs(y, rot, inter):
    """|a| + |b| of each channel's pair (|y| where nothing turns)."""
    s = np.abs(y)
    a, b = B.rotation_pairs(rot, inter)
    s[..., a] = s[..., b] = s[..., a] + s[..., b]
    return s


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", QK)
def test_qk_norm_rope_and_backward(A, T, Hq, Hk, D, rot, inter, dt):
    q, k, gains, pos, freq = _qk_inputs(T, Hq, Hk, D, rot, dt, 1)
    g = _gen(2)
    gq, gk = _randn(g, T, Hq, D, dtype=dt), _randn(g, T, Hk, D, dtype=dt)
    rope = dict(positions=pos, inv_freq=freq) if rot else {}
    outs = [torch.full((T, h, D), float("nan"), dtype=dt, device="cuda") for h in (Hq, Hk)]
    A.attnres_qk_norm_rope(q, k, *outs, q_gain=gains[0], k_gain=gains[1], interleaved=inter, **rope)
    grads = [torch.full((T, h, D), float("nan"), dtype=dt, device="cuda") for h in (Hq, Hk)]
    dgs = [torch.empty(D, device="cuda") for _ in range(2)]
    A.attnres_qk_norm_rope_backward(q, k, gq, gk, *grads, q_gain=gains[0], k_gain=gains[1], grad_q_gain=dgs[0],
                                    grad_k_gain=dgs[1], interleaved=inter, **rope)
    p64, f64 = to64(pos), to64(freq)
    for x, gain, go, out, dx, dg in zip((q, k), gains, (gq, gk), outs, grads, dgs):
        x64, gain64, go64 = to64(x), to64(gain), to64(go)
        y = B.qk_norm_rope(x64, gain64, p64, f64, inter, 1e-5)
        # norm: a sum of D squares under a root (half its error) and 6 operations; the angle: reduced to
        # half a turn with 2^-24 of a turn's error, i.e. 4 e of the pair, and cos, sin within 4 e
        flat = B.qk_norm_rope(x64, gain64, p64, np.zeros(0), inter, 1e-5)
        pair = _pair_abs(flat, rot, inter)
        _close(out, y, U[dt] * np.abs(y) + (D / 2 + 24) * E * pair, "out")
        wdx, wdg = B.qk_norm_rope_backward(x64, gain64, p64, f64, inter, 1e-5, go64)
        rho = np.sqrt((x64 * x64).mean(-1, keepdims=True) + 1e-5)
        hat = np.abs(x64) / rho
        n = _pair_abs(go64, rot, inter) * np.abs(gain64)
        cond = (n + hat * (n * hat).mean(-1, keepdims=True)) / rho
        _close(dx, wdx, U[dt] * np.abs(wdx) + (2 * D + 48) * E * cond, "grad_x")
        ndg = (_pair_abs(go64, rot, inter) * hat).sum((0, 1))
        _close(dg, wdg, (D / 2 + 24 + x64.shape[0] * x64.shape[1]) * E * ndg, "grad_gain")


@pytest.mark.parametrize("far", [1 << 20, (1 << 24) - 2500, (1 << 31) + 12345, -3000])
def test_far_positions_keep_their_angle(A, far):
    q, k, _, pos, freq = _qk_inputs(40, 2, 1, 64, 64, torch.float32, 4, far)
    outs = [torch.empty_like(q), torch.empty_like(k)]
    A.attnres_qk_norm_rope(q, k, *outs, positions=pos, inv_freq=freq)
    for x, out in zip((q, k), outs):
        want = B.qk_norm_rope(to64(x), None, to64(pos), to64(freq), False, 1e-5)
        pair = _pair_abs(B.qk_norm_rope(to64(x), None, to64(pos), np.zeros(0), False, 1e-5), 64, False)
        _close(out, want, U[torch.float32] * np.abs(want) + (32 + 24) * E * pair, far)


@pytest.mark.parametrize("D,rot", [(128, 128), (37, 12)])
def test_qk_norm_rope_in_place_and_one_of_two(A, D, rot):
    dt = torch.bfloat16
    q, k, gains, pos, freq = _qk_inputs(50, 6, 2, D, rot, dt, 7)
    kw = dict(positions=pos, inv_freq=freq)
    want = [torch.empty_like(q), torch.empty_like(k)]
    A.attnres_qk_norm_rope(q, k, *want, q_gain=gains[0], k_gain=gains[1], **kw)
    only = torch.empty_like(k)
    A.attnres_qk_norm_rope(None, k, None, only, k_gain=gains[1], **kw)
    assert torch.equal(only, want[1])
    rows = torch.zeros(50, 10 * D, dtype=dt, device="cuda")  # q, k, v side by side
    q2, k2 = rows[:, :6 * D].unflatten(1, (6, D)), rows[:, 6 * D:8 * D].unflatten(1, (2, D))
    q2.copy_(q)
    k2.copy_(k)
    A.attnres_qk_norm_rope(q2, k2, q2, k2, q_gain=gains[0], k_gain=gains[1], **kw)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1]) and not rows[:, 8 * D:].any()


def test_qk_norm_rope_zero_rows_and_no_tokens(A):
    z = torch.zeros(3, 2, 64, device="cuda")
    out = torch.full_like(z, float("nan"))
    A.attnres_qk_norm_rope(z, None, out, None)
    assert not out.any()
    dg = torch.full((64,), float("nan"), device="cuda")
    A.attnres_qk_norm_rope_backward(z[:0], None, z[:0], None, out[:0], None, grad_q_gain=dg)
    assert not dg.any()
    A.attnres_qk_norm_rope(z[:0], None, out[:0], None)


# -------------------------------------------------------- linear attention --

ATT = [  # T, sequences, H, Dk, Dv
    (1, 1, 1, 8, 8), (5, 1, 2, 64, 64), (128, 1, 2, 128, 128), (129, 1, 3, 128, 128), (300, 4, 2, 128, 64), (257, 3, 2, 64, 128),
    (700, 9, 1, 64, 64), (1000, 1, 1, 128, 128), (200, 30, 2, 128, 128), (77, 3, 2, 96, 160), (70, 2, 1, 37, 5), (50, 2, 2, 1, 256),
    (90, 1, 1, 256, 33),
    (2000, 1, 2, 128, 128), (4100, 5, 1, 64, 128), (3001, 3, 2, 40, 24),  # long enough to be cut into pieces
    (300, 4, 2, 96, 96), (2000, 2, 2, 96, 80), (500, 3, 2, 32, 112), (140, 2, 1, 16, 16), (3001, 3, 2, 80, 48),
]


def _att_inputs(T, n, H, Dk, Dv, dt, seed, initial=True):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.sort(r.integers(0, T + 1, n - 1)), [T]]).astype(np.int32)  # empty ones among them
    g = _gen(seed)
    rows = _randn(g, T, H * (2 * Dk + Dv), dtype=dt)
    q, k = rows[:, :H * Dk].unflatten(1, (H, Dk)), rows[:, H * Dk:2 * H * Dk].unflatten(1, (H, Dk))
    v = rows[:, 2 * H * Dk:].unflatten(1, (H, Dv))
    decay = -torch.exp2(-6.0 * torch.rand(H, generator=g, device="cuda"))
    if H > 2:
        decay[0], decay[1] = 0.0, -200.0  # nothing forgotten; everything at once
    s0 = _randn(g, n, H, Dk, Dv) if initial else None
    return q, k, v, decay, torch.from_numpy(cu).cuda(), s0


def _att_tol(T, Dk, Dv, dt):
    """Relative to the sums over absolute values: fp32 sums over the channels
    and the tokens (32 operations more for powers, scales and joins); with
    bf16 tensors the scores and the state each enter a product rounded."""
    return (Dk + Dv + T + 64) * E + (2 * U[dt] if dt == torch.bfloat16 else 0)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,n,H,Dk,Dv", ATT)
def test_linear_attention(A, T, n, H, Dk, Dv, dt):
    for initial in (False, True):
        q, k, v, decay, cu, s0 = _att_inputs(T, n, H, Dk, Dv, dt, 3, initial)
        out = torch.full((T, H, Dv), float("nan"), dtype=dt, device="cuda")
        fin = torch.full((n, H, Dk, Dv), float("nan"), device="cuda")
        err = _err()
        A.attnres_linear_attention(q, k, v, decay, out, cu_seqlens=cu, initial_state=s0, final_state=fin, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        args = [to64(t) for t in (q, k, v)]
        s64, scale = None if s0 is None else to64(s0), Dk ** -0.5
        want, wfin = B.linear_attention(*args, to64(decay), to64(cu).astype(int), s64, scale)
        cond, cfin = B.linear_attention(*[np.abs(t) for t in args], to64(decay), to64(cu).astype(int),
                                        None if s64 is None else np.abs(s64), scale)
        _close(out, want, U[dt] * np.abs(want) + _att_tol(T, Dk, Dv, dt) * cond, "out")
        _close(fin, wfin, (T + 64) * E * cfin, "final state")
        if initial:  # the state carried on in place: the same bits
            out2 = torch.empty_like(out)
            A.attnres_linear_attention(q, k, v, decay, out2, cu_seqlens=cu, initial_state=s0, final_state=s0)
            assert torch.equal(out2, out) and torch.equal(s0, fin)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,n,H,Dk,Dv", ATT)
def test_linear_attention_backward(A, T, n, H, Dk, Dv, dt):
    for initial in (False, True):
        q, k, v, decay, cu, s0 = _att_inputs(T, n, H, Dk, Dv, dt, 5, initial)
        g = _gen(6)
        do = _randn(g, T, H, Dv, dtype=dt)
        ds1 = _randn(g, n, H, Dk, Dv) if initial else None
        grads = [torch.full((T, H, w), float("nan"), dtype=dt, device="cuda") for w in (Dk, Dk, Dv)]
        ds0 = torch.full((n, H, Dk, Dv), float("nan"), device="cuda")
        err = _err()
        A.attnres_linear_attention_backward(q, k, v, decay, do, *grads, cu_seqlens=cu, initial_state=s0,
                                            grad_final_state=ds1, grad_initial_state=ds0, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        x = [to64(t) for t in (q, k, v)]
        cu64, d64 = to64(cu).astype(int), to64(decay)
        s64, r64 = (None, None) if not initial else (to64(s0), to64(ds1))
        want = B.linear_attention_backward(*x, d64, cu64, s64, Dk ** -0.5, to64(do), r64)
        cond = B.linear_attention_backward(*[np.abs(t) for t in x], d64, cu64, None if s64 is None else np.abs(s64), Dk ** -0.5,
                                           np.abs(to64(do)), None if r64 is None else np.abs(r64))
        for got, w, c, name in zip(grads, want, cond, ("dq", "dk", "dv")):
            _close(got, w, U[dt] * np.abs(w) + _att_tol(T, Dk, Dv, dt) * c, name)
        _close(ds0, want[3], (T + 64) * E * cond[3], "grad_initial_state")
        if initial:
            A.attnres_linear_attention_backward(q, k, v, decay, do, *grads, cu_seqlens=cu, initial_state=s0,
                                                grad_final_state=ds1, grad_initial_state=ds1)
            assert torch.equal(ds1, ds0)


@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 40)])
def test_rows_outside_every_sequence_stay_and_do_not_matter(A, dt, D):
    """Rows before the first, between no sequences and behind the last: not
    written, and neither their infinities nor their NaN reach a result."""
    T, H = 400, 2
    q, k, v, decay, _, s0 = _att_inputs(T, 2, H, D, D, dt, 9)
    cu = torch.tensor([10, 150, 333], dtype=torch.int32, device="cuda")
    q, k, v = q.clone(), k.clone(), v.clone()
    do = _randn(_gen(1), T, H, D, dtype=dt)

    def run():
        outs = [torch.full((T, H, D), 7.0, dtype=dt, device="cuda") for _ in range(4)]
        st = [torch.empty_like(s0) for _ in range(2)]
        A.attnres_linear_attention(q, k, v, decay, outs[0], cu_seqlens=cu, initial_state=s0, final_state=st[0])
        A.attnres_linear_attention_backward(q, k, v, decay, do, *outs[1:], cu_seqlens=cu, initial_state=s0,
                                            grad_final_state=s0, grad_initial_state=st[1])
        return outs, st
    a, sa = run()
    for t in (q, k, v, do):
        t[:10] = float("nan")
        t[333:] = float("inf")
    b, sb = run()
    for x, y in zip(a + sa, b + sb):
        assert torch.equal(x, y)
    for x in b:
        assert (x[:10] == 7).all() and (x[333:] == 7).all() and torch.isfinite(x).all()


def test_one_sequence_does_not_reach_another(A):
    """NaN in one sequence of a batch stays there."""
    q, k, v, decay, _, s0 = _att_inputs(300, 3, 2, 128, 128, torch.bfloat16, 2)
    cu = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda")
    q, k, v = q.clone(), k.clone(), v.clone()
    out, fin = torch.empty_like(v), torch.empty_like(s0)
    A.attnres_linear_attention(q, k, v, decay, out, cu_seqlens=cu, initial_state=s0, final_state=fin)
    for t in (q, k, v):
        t[100:200] = float("nan")
    out2, fin2 = torch.empty_like(out), torch.empty_like(fin)
    A.attnres_linear_attention(q, k, v, decay, out2, cu_seqlens=cu, initial_state=s0, final_state=fin2)
    keep = [*range(100), *range(200, 300)]
    assert torch.equal(out[keep], out2[keep]) and torch.equal(fin[[0, 2]], fin2[[0, 2]])
    assert torch.isnan(out2[100:200]).all() and torch.isnan(fin2[1]).all()


@pytest.mark.parametrize("dt,D,T", [(torch.bfloat16, 128, 300), (torch.bfloat16, 64, 6000), (torch.bfloat16, 96, 300), (torch.float32, 40, 150),
                                    (torch.bfloat16, 24, 6000)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_no_token_reaches_an_earlier_one(A, dt, D, T, bad):
    """Infinities and NaN of a token behind: the outputs before it, and the
    gradients that do not depend on it, are the formula's."""
    t, H = T - 30, 2
    q, k, v, decay, _, s0 = _att_inputs(T, 1, H, D, D, dt, 16)
    q, k, v, do = q.clone(), k.clone(), v.clone(), _randn(_gen(17), T, H, D, dtype=dt)
    x, do64 = [to64(a[:t]) for a in (q, k, v)], to64(do)
    want, _ = B.linear_attention(*x, to64(decay), [0, t], to64(s0), D ** -0.5)
    cond, _ = B.linear_attention(*[np.abs(a) for a in x], to64(decay), [0, t], np.abs(to64(s0)), D ** -0.5)
    # dk and dv run backwards: what comes before token u does not reach them
    u = 31
    y = [to64(a[u:]) for a in (q, k, v)]
    back = B.linear_attention_backward(*y, to64(decay), [0, T - u], None, D ** -0.5, do64[u:], None)
    cback = B.linear_attention_backward(*[np.abs(a) for a in y], to64(decay), [0, T - u], None, D ** -0.5, np.abs(do64[u:]), None)
    for a in (q, k, v):
        a[t] = bad
        a[t + 7, 1, 3] = -bad
    out, fin = torch.empty_like(do), torch.empty_like(s0)
    A.attnres_linear_attention(q, k, v, decay, out, initial_state=s0, final_state=fin)
    _close(out[:t], want, U[dt] * np.abs(want) + _att_tol(T, D, D, dt) * cond, "out")
    assert not torch.isfinite(out[t:, 1]).any()
    q, k, v, _, _, _ = _att_inputs(T, 1, H, D, D, dt, 16)
    q, k, v = q.clone(), k.clone(), v.clone()
    for a in (q, k, v, do):
        a[u - 1] = bad
        a[u - 9, 1, 3] = -bad
    grads = [torch.empty_like(do) for _ in range(3)]
    A.attnres_linear_attention_backward(q, k, v, decay, do, *grads)
    for got, w, c, name in zip(grads[1:], back[1:3], cback[1:3], ("dk", "dv")):
        _close(got[u:], w, U[dt] * np.abs(w) + _att_tol(T, D, D, dt) * c, name)


def test_a_state_survives_no_tokens(A):
    s0 = torch.randn(2, 3, 64, 64, device="cuda")
    e = torch.empty(0, 3, 64, device="cuda", dtype=torch.bfloat16)
    cu, fin, g = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.empty_like(s0), torch.zeros(3, device="cuda")
    A.attnres_linear_attention(e, e, e, g, e, cu_seqlens=cu, initial_state=s0, final_state=fin)
    assert torch.equal(fin, s0)
    A.attnres_linear_attention(e, e, e, g, e, cu_seqlens=cu, final_state=fin)
    assert not fin.any()
    A.attnres_linear_attention_backward(e, e, e, g, e, e, e, e, cu_seqlens=cu, grad_final_state=s0, grad_initial_state=fin)
    assert torch.equal(fin, s0)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("b,slots,H,Dk,Dv", [(1, 1, 1, 1, 1), (1, 4, 56, 128, 128), (64, 70, 4, 128, 128), (9, 9, 3, 37, 5),
                                             (5, 8, 2, 256, 256), (33, 40, 2, 64, 96), (300, 301, 1, 64, 64)])
def test_linear_attention_step(A, b, slots, H, Dk, Dv, dt):
    g = _gen(8)
    rows = _randn(g, b, H * (2 * Dk + Dv), dtype=dt)
    q, k = rows[:, :H * Dk].unflatten(1, (H, Dk)), rows[:, H * Dk:2 * H * Dk].unflatten(1, (H, Dk))
    v = rows[:, 2 * H * Dk:].unflatten(1, (H, Dv))
    decay, state = -torch.rand(H, generator=g, device="cuda"), _randn(g, slots, H, Dk, Dv)
    at = torch.randperm(slots, generator=g, device="cuda")[:b].int()
    if b >= 9:
        at[2], at[4], at[7] = at[0], -1, at[0]  # one sequence's three tokens, and a padding row
        at[5] = slots
    ident = b % 2 == 1 and b < 9
    st, out = state.clone(), torch.full((b, H, Dv), 7.0, dtype=dt, device="cuda")
    A.attnres_linear_attention_step(q, k, v, decay, st, out, slots=None if ident else at)
    sl = list(range(b)) if ident else at.tolist()
    x = [to64(t) for t in (q, k, v)]
    want, wst = B.linear_attention_step(*x, to64(decay), to64(state), sl, Dk ** -0.5)
    cond, cst = B.linear_attention_step(*[np.abs(t) for t in x], to64(decay), np.abs(to64(state)), sl, Dk ** -0.5)
    live = ~np.isnan(want).any(axis=(1, 2))
    assert (out[torch.from_numpy(~live).cuda()] == 7).all()
    _close(out[torch.from_numpy(live).cuda()], want[live], (U[dt] * np.abs(want) + (Dk + 32) * E * cond)[live], "out")
    _close(st, wst, 8 * E * cst, "state")


def test_steps_go_on_from_a_prompt(A):
    """A prompt, then its next tokens one by one, against all of it at once
    (the state is fp32 in both; bf16 scores in the prompt's form only)."""
    T, P, H, D = 200, 150, 4, 128
    q, k, v, decay, _, _ = _att_inputs(T, 1, H, D, D, torch.bfloat16, 11)
    out, fin = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, H, D, D, device="cuda")
    A.attnres_linear_attention(q[:P], k[:P], v[:P], decay, out[:P], final_state=fin)
    for t in range(P, T):
        A.attnres_linear_attention_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], decay, fin, out[t:t + 1])
    x = [to64(t) for t in (q, k, v)]
    want, wfin = B.linear_attention(*x, to64(decay), [0, T], None, D ** -0.5)
    cond, cfin = B.linear_attention(*[np.abs(t) for t in x], to64(decay), [0, T], None, D ** -0.5)
    _close(out, want, U[torch.bfloat16] * np.abs(want) + _att_tol(T, D, D, torch.bfloat16) * cond, "out")
    _close(fin, wfin, (T + 64) * E * cfin, "state")


def test_bad_offsets_are_clamped(A):
    """Offsets outside 0..T read and write nothing outside the tensors."""
    q, k, v, decay, _, _ = _att_inputs(60, 1, 2, 64, 64, torch.bfloat16, 12)
    cu = torch.tensor([-5, 20, 90], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 20, 60], dtype=torch.int32, device="cuda")
    a, b = torch.empty(60, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(60, 2, 64, dtype=torch.bfloat16, device="cuda")
    A.attnres_linear_attention(q, k, v, decay, a, cu_seqlens=cu)
    A.attnres_linear_attention(q, k, v, decay, b, cu_seqlens=good)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 64), (torch.float32, 24)])
def test_offsets_that_decrease_stay_inside(A, dt, D):
    """What they select is not defined, but nothing outside the rows is
    written, and the call returns (long enough to run in pieces)."""
    T, H = 4100, 2
    cu = torch.tensor([0, 4000, 100, 4100, 50, 4100, 0], dtype=torch.int32, device="cuda")
    assert A.attnres_linear_attention_workspace_size(T, H, D, D, dt, 6) > 0
    rows = _randn(_gen(18), T, 3 * H * D, dtype=dt)
    q, k, v = (rows[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in range(3))
    decay, fin = torch.full((H,), -0.01, device="cuda"), torch.zeros(8, H, D, D, device="cuda")
    outs = [torch.full((T + 256, H, D), 7.0, dtype=dt, device="cuda") for _ in range(4)]
    views = [o[128:T + 128] for o in outs]
    err = _err()
    A.attnres_linear_attention(q, k, v, decay, views[0], cu_seqlens=cu, final_state=fin[1:7], dev_err=err)
    A.attnres_linear_attention_backward(q, k, v, decay, v, *views[1:], cu_seqlens=cu, grad_initial_state=fin[1:7], dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not fin[0].any() and not fin[7].any()
    for o in outs:
        assert (o[:128] == 7).all() and (o[T + 128:] == 7).all()


@pytest.mark.parametrize("dt,T,n,H,D", [(torch.bfloat16, 300, 4, 3, 128), (torch.bfloat16, 9000, 3, 1, 64),
                                        (torch.float32, 300, 4, 3, 40), (torch.float32, 6000, 3, 1, 24)])
def test_a_decay_that_leaves_nothing(A, dt, T, n, H, D):
    """log_decay = -inf is a decay of 0, which -200 rounds to in fp32: the
    same bits, in one piece and in several, with an empty sequence."""
    q, k, v, _, cu, s0 = _att_inputs(T, n, H, D, D, dt, 13)
    cu[1] = cu[2]
    do = _randn(_gen(14), T, H, D, dtype=dt)
    runs = []
    for value in (-200.0, float("-inf")):
        decay = torch.full((H,), value, device="cuda")
        outs = [torch.empty(T, H, D, dtype=dt, device="cuda") for _ in range(4)]
        st = [torch.empty_like(s0) for _ in range(2)]
        A.attnres_linear_attention(q, k, v, decay, outs[0], cu_seqlens=cu, initial_state=s0, final_state=st[0])
        A.attnres_linear_attention_backward(q, k, v, decay, do, *outs[1:], cu_seqlens=cu, initial_state=s0, grad_final_state=s0,
                                            grad_initial_state=st[1])
        o, pool = torch.empty(n, H, D, dtype=dt, device="cuda"), s0.clone()
        A.attnres_linear_attention_step(q[:n], k[:n], v[:n], decay, pool, o)
        runs.append([*outs, *st, o, pool])
    for a, b in zip(*runs):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 24])
def test_no_workspace_is_used_where_none_is_given(A, D):
    """A NULL workspace has no bytes whatever its size argument says, and
    tensors off the 16-byte boundaries, for which none is asked, do without."""
    from depth_wise_attention_block_gb300 import _native as N
    T, H, dt = 700, 1, torch.bfloat16
    assert A.attnres_linear_attention_workspace_size(T, H, 64, 64, dt) == 0 or D != 64
    wide = _randn(_gen(15), T, 3 * D + 1, dtype=dt)
    q, k, v = (wide[:, 1 + i * D:1 + (i + 1) * D].unflatten(1, (H, D)) for i in range(3))
    decay = torch.full((H,), -0.01, device="cuda")
    want, got = (torch.empty(T, H, D, dtype=dt, device="cuda") for _ in range(2))
    A.attnres_linear_attention(q, k, v, decay, want)
    need = A.attnres_linear_attention_workspace_size(T, H, D, D, dt)
    s = 3 * D + 1
    rc = N.lib.attnres_linear_attention(q.data_ptr(), s, k.data_ptr(), s, v.data_ptr(), s, T, H, D, D, 1, decay.data_ptr(), None, 1, None,
                                        None, D ** -0.5, got.data_ptr(), D, None, 1 << 40, None,
                                        torch.cuda.current_stream().cuda_stream)
    if need > 0:
        assert rc == N.ATTNRES_EINVAL
    else:
        assert rc == 0 and torch.equal(want, got)


def test_a_stride_of_a_single_row_does_not_matter(A):
    from depth_wise_attention_block_gb300 import _native as N
    x, w, _, _ = _linear_inputs(1, 264, 136, torch.bfloat16, 23)
    want, got = torch.empty(1, 264, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 264, dtype=torch.bfloat16, device="cuda")
    A.attnres_linear(x, w, want)
    rc = N.lib.attnres_linear(x.data_ptr(), 1 << 41, w.data_ptr(), None, None, 264, got.data_ptr(), 1 << 41, 1, 264, 136, 1, 0, None, 0,
                              None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(want, got)


def test_gain_gradient_of_no_heads_is_zero(A):
    q = torch.randn(5, 2, 64, device="cuda")
    none, dg, dk = torch.empty(5, 0, 64, device="cuda"), torch.empty(64, device="cuda"), torch.full((64,), 7.0, device="cuda")
    A.attnres_qk_norm_rope_backward(q, none, q, none, torch.empty_like(q), none, grad_q_gain=dg, grad_k_gain=dk)
    assert not dk.any() and torch.isfinite(dg).all() and dg.any()


# ---------------------------------------------------------------- together --

def test_other_streams_and_repeats_give_the_same_bits(A):
    x, w, b, res = _linear_inputs(200, 264, 136, torch.bfloat16, 21)
    q, k, v, decay, cu, s0 = _att_inputs(500, 3, 4, 128, 128, torch.bfloat16, 22)

    def run(stream=None):
        out, gx, gw, gb = torch.empty_like(res), torch.empty_like(x), torch.empty_like(w), torch.empty(264, device="cuda")
        o, fin = torch.empty(500, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty_like(s0)
        gr = [torch.empty(500, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        A.attnres_linear(x, w, out, bias=b, residual=res, activation="silu", stream=stream)
        A.attnres_linear_backward(x, w, res, gx, gw, gb, bias=b, activation="silu", stream=stream)
        A.attnres_linear_attention(q, k, v, decay, o, cu_seqlens=cu, initial_state=s0, final_state=fin, stream=stream)
        A.attnres_linear_attention_backward(q, k, v, decay, o, *gr, cu_seqlens=cu, initial_state=s0, stream=stream)
        torch.cuda.synchronize()
        return [out, gx, gw, gb, o, fin, *gr]
    first = run()
    side = torch.cuda.Stream()
    for other in (run(), run(side), run(side.cuda_stream)):
        for a, c in zip(first, other):
            assert torch.equal(a, c)
