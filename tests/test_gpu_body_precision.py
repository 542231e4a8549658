"""Bars that a lost term does not pass: inputs whose errors do not average out,
or whose sums are short, so that the bound of the arithmetic lies well below
what a term of fewer bits would cost.  E = 2^-23 bounds one fp32 operation or
one truncated step of an accumulator, U half a rounding step of the stored type
(bf16 2^-8, fp32 2^-24).
"""
import math

import numpy as np
import pytest
import torch

from oracle import body_oracle as B

E = 2.0 ** -23
UB = 2.0 ** -8
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def to64(t):
    return t.detach().double().cpu().numpy()


def _randn(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# ------------------------------------------------- fp32 products, three terms --

# 1 + 2^-8 + 2^-15 + 63/64 2^-16: cut to 8 bits it leaves 2^-8 + .., which
# rounded to 8 bits leaves all but 2^-16.  As operand of every product of a sum
# of one sign it makes each of the six products of terms worth 2^-16.1 or more of
# the result, none of which averages out; a sum over 16 steps may be off by
# (16 + 16) 2^-23 = 2^-18.
PATTERN = 1 + 2.0 ** -8 + 2.0 ** -15 + 63 / 64 * 2.0 ** -16
SHORT = 16
SUM_BAR = (SHORT + 16) * E + 2.0 ** -24


def _rows(seed, rows, cols, dev):
    """PATTERN times powers of two, by rows: every sum has one size of addends."""
    p = torch.randint(-3, 4, (rows, 1), generator=torch.Generator().manual_seed(seed)).double().exp2() * PATTERN
    return p.expand(rows, cols).float().contiguous().to(dev)


def _round_bits(v):
    """v rounded to 8 significant bits (nearest, ties to even)."""
    m, e = math.frexp(v)
    return math.ldexp(round(m * 256), e - 8)


def test_the_pattern_shows_each_term():
    """On the CPU: the product without any one of the six leading products of
    terms misses the bar at least threefold, and with them meets it."""
    assert float(np.float32(PATTERN)) == PATTERN
    hi = math.floor(PATTERN * 128) / 128
    mid = _round_bits(PATTERN - hi)
    lo = _round_bits(PATTERN - hi - mid)
    t = {"h": hi, "m": mid, "l": lo}
    exact = PATTERN * PATTERN
    six = ["hh", "hm", "mh", "mm", "hl", "lh"]
    whole = sum(t[a] * t[b] for a, b in six)
    assert abs(whole / exact - 1) <= SUM_BAR / 4
    for gone in six:
        assert abs((whole - t[gone[0]] * t[gone[1]]) / exact - 1) >= 3 * SUM_BAR, gone


# wide tiles, clusters, and few rows whose weights are split on the way in
# (short products: large enough for the tensor cores)
@gpu
@pytest.mark.parametrize("m,n", [(1024, 1024), (16, 65536), (64, 16384), (128, 8192), (200, 6000)])
def test_fp32_products_keep_every_term(A, m, n):
    x, w = _rows(1, m, SHORT, "cuda"), _rows(2, n, SHORT, "cuda")
    out = torch.empty(m, n, device="cuda")
    A.attnres_linear(x, w, out)
    want = x.double() @ w.double().T
    assert ((out.double() / want - 1).abs() <= SUM_BAR).all()


@gpu
@pytest.mark.parametrize("rows", [128, 1024, 5000])
def test_fp32_gradients_keep_every_term(A, rows):
    """grad_x over 16 outputs, grad_w over 16 tokens: MN-major operands."""
    gx = torch.empty(rows, 512, device="cuda")
    w = _rows(3, 1, SHORT, "cuda").T.contiguous().expand(SHORT, 512).contiguous()
    g, x = _rows(4, rows, SHORT, "cuda"), torch.zeros(rows, 512, device="cuda")
    A.attnres_linear_backward(x, w, g, gx)
    assert ((gx.double() / (g.double() @ w.double()) - 1).abs() <= SUM_BAR).all()
    gw = torch.empty(rows, 512, device="cuda")
    g = _rows(5, rows, SHORT, "cuda").T.contiguous()
    x, w = _rows(6, 1, 512, "cuda").expand(SHORT, 512).contiguous(), torch.zeros(rows, 512, device="cuda")
    A.attnres_linear_backward(x, w, g, None, gw)
    assert ((gw.double() / (g.double().T @ x.double()) - 1).abs() <= SUM_BAR).all()


# ------------------------------------------------------- states, three terms --

@gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Dk,Dv", [(128, 128, 128), (150, 128, 64), (100, 64, 128), (6000, 128, 128), (6000, 64, 64), (300, 80, 96)])
def test_states_keep_24_bits(A, dt, T, Dk, Dv):
    """One token per channel of k: every entry of the state is one product,
    decayed.  A power's error is that of exp (2 ulp) and of its argument, at
    most 1 here; the product and the sum of its terms take 4 operations, each
    chunk that the entry passes (of at least 64 tokens), and a join of pieces,
    a power and an addition.  Two bf16 terms of a weighted key would leave up
    to 2^-16 of it, more than this bar in a good part of the thousands of
    entries."""
    H = 2
    tail = min(T, 2 * Dk)
    k = torch.zeros(T, H, Dk, device="cuda", dtype=dt)
    at = T - tail + torch.arange(Dk, device="cuda") * (tail // Dk)
    k[at, :, torch.arange(Dk, device="cuda")] = (1 + _randn(1, Dk, H).abs()).to(dt)
    v, q = _randn(2, T, H, Dv, dtype=dt), _randn(3, T, H, Dk, dtype=dt)
    decay = -torch.tensor([1.0, 0.7], device="cuda") / (2 * Dk)
    out, fin = torch.empty_like(v), torch.empty(1, H, Dk, Dv, device="cuda")
    A.attnres_linear_attention(q, k, v, decay, out, final_state=fin)
    gone = (T - 1 - at).double()
    power = torch.exp(decay.double()[:, None] * gone)                                # [H, Dk]
    want = (power * k[at, :, torch.arange(Dk, device="cuda")].double().T)[..., None] * v[at].double().transpose(0, 1)
    rel = (fin[0].double() / want - 1)
    bar = (3 + 4 + 4 * (1 + math.ceil(tail / 64)) + 4) * E
    assert bar < 2.0 ** -18
    assert (rel.abs() <= bar).all(), float(rel.abs().max() / bar)
    # the gradient of the initial state, from the other end: d0 = exp(g) R, R the decayed sum of scale q do^T
    do = torch.zeros(T, H, Dv, device="cuda", dtype=dt)
    n = min(Dv, tail)
    first = torch.arange(n, device="cuda")
    do[first, :, first] = (1 + _randn(4, n, H).abs()).to(dt)
    grads = [torch.empty_like(q), torch.empty_like(q), torch.empty_like(v)]
    d0 = torch.empty_like(fin)
    A.attnres_linear_attention_backward(q, k, v, decay, do, *grads, grad_initial_state=d0, scale=1.0)
    power = torch.exp(decay.double()[:, None] * (first + 1).double())                # [H, n]
    want = q[first].double().permute(1, 2, 0) * (power * do[first, :, first].double().T)[:, None, :]
    rel = d0[0, :, :, :n].double() / want - 1
    assert (rel.abs() <= bar).all(), float(rel.abs().max() / bar)


# --------------------------- bf16 attention: scores and state in two terms -----

def _att(T, n, H, Dk, Dv, seed, initial):
    q, k, v, do = (_randn(seed + i, T, H, D, dtype=torch.bfloat16) for i, D in enumerate((Dk, Dk, Dv, Dv)))
    return q, k, v, do, _randn(seed + 4, n, H, Dk, Dv) if initial else None


def _score_part(a, b, g, cu, reverse, chunk=128):
    """What of a row's scores lies in its own chunk of its own sequence: the
    mask [T, T] (a sequence's chunks begin at its start, reversed ones at its end)."""
    T = a.shape[0]
    mask = np.zeros((T, T), bool)
    for s, e in zip(cu[:-1], cu[1:]):
        i = np.arange(s, e)
        c = (e - 1 - i) // chunk if reverse else (i - s) // chunk
        ago = i[None, :] - i[:, None] if reverse else i[:, None] - i[None, :]
        mask[s:e, s:e] = (c[:, None] == c[None, :]) & (ago >= 0)
    return mask


def _conds(a, b, c, g, cu, scale, reverse, mask):
    """Sums over absolute values of a row's result, in its chunk and from before
    it (without an initial state)."""
    T, H = a.shape[:2]
    i = np.arange(T)
    ago = (i[None, :] - i[:, None]) if reverse else (i[:, None] - i[None, :])
    seq = np.searchsorted(cu[1:], i, side="right")
    live = (ago >= 0) & (seq[:, None] == seq[None, :])
    inside, before = np.zeros((T, H, c.shape[2])), np.zeros((T, H, c.shape[2]))
    for h in range(H):
        P = scale * (np.abs(a[:, h]) @ np.abs(b[:, h]).T) * np.where(live, np.exp(g[h] * np.where(live, ago, 0)), 0.0)
        inside[:, h] = np.where(mask, P, 0) @ np.abs(c[:, h])
        before[:, h] = np.where(mask, 0, P) @ np.abs(c[:, h])
    return inside, before


@gpu
@pytest.mark.parametrize("T,cu,Dk,Dv", [
    (128, (0, 128), 128, 128), (97, (0, 40, 97), 64, 64), (128, (0, 1, 128), 96, 48), (500, (0, 130, 500), 128, 64),
    (3000, (0, 1100, 3000), 64, 128), (3000, (0, 3000), 128, 128)])
def test_bf16_attention_rounds_once(A, T, cu, Dk, Dv):
    """The scores of the chunk and the state from those before as two bf16 terms
    each (2^-16 of them), the state's own sums with at least 16 bits, and the
    output's own rounding.  One term of either would miss by up to 2^-8 of its
    sums, 100 times their share of this bar."""
    H = 2
    q, k, v, do, _ = _att(T, len(cu) - 1, H, Dk, Dv, 10, False)
    g = -torch.tensor([0.003, 0.05], device="cuda")
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out, grads = torch.empty_like(v), [torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)]
    A.attnres_linear_attention(q, k, v, g, out, cu_seqlens=cut)
    A.attnres_linear_attention_backward(q, k, v, g, do, *grads, cu_seqlens=cut)
    q64, k64, v64, do64, g64 = (to64(t) for t in (q, k, v, do, g))
    scale = Dk ** -0.5
    want = [B.linear_attention(q64, k64, v64, g64, cu, None, scale)[0],
            *B.linear_attention_backward(q64, k64, v64, g64, cu, None, scale, do64, None)[:3]]
    scans = [(q64, k64, v64, False), (do64, v64, k64, False), (v64, do64, q64, True), (k64, q64, do64, True)]
    fp32 = (Dk + Dv + T + 64) * E
    for name, got, ref, (a, b, c, rev) in zip(("out", "dq", "dk", "dv"), [out, *grads], want, scans):
        inside, before = _conds(a, b, c, g64, np.array(cu), scale, rev, _score_part(a, b, g64, cu, rev))
        bound = UB * np.abs(ref) + (2.0 ** -16 + fp32) * (inside + 2 * before) + 2.0 ** -129
        err = np.abs(to64(got) - ref)
        assert (err <= bound).all(), (name, float((err / bound).max()))


# --------------------------------------------- activations far from zero -------

@gpu
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("shape", ["few rows", "many rows", "small"])
def test_fp32_activations_keep_their_digits_far_out(A, act, shape):
    """z itself exact (one product with 1), from -9 to 9: relative to the value.
    An activation's value and slope at z are those of z (1 + a few 2^-24), which
    the exponent z^2 / 2 (gelu), 0.8 (z + 0.045 z^3) (tanh gelu, both doubled) or
    z (silu) multiplies; 16 operations more."""
    z = torch.linspace(-9, 9, 1537, device="cuda")
    z = z[(z.abs() > 1e-3)]
    m = {"few rows": 64, "many rows": 2048, "small": 4}[shape]
    n = {"few rows": 4096, "many rows": 2048, "small": 4}[shape]
    k = 4 if shape == "small" else 128
    x, w = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
    x[:, 0] = z[torch.arange(m, device="cuda") * 37 % z.numel()] if shape != "small" else torch.tensor([-8.5, -5.0, -3.0, 4.0], device="cuda")
    w[:, 0] = 1
    out = torch.empty(m, n, device="cuda")
    A.attnres_linear(x, w, out, activation=act)
    z64 = to64(x[:, 0])
    erfc = np.vectorize(math.erfc)
    c = math.sqrt(2 / math.pi)
    u2 = 2 * c * (z64 + 0.044715 * z64 ** 3)
    sig = lambda t: 1 / (1 + np.exp(-t))
    value, slope, grow = {
        "gelu": (z64 * 0.5 * erfc(-z64 / math.sqrt(2)),
                 0.5 * erfc(-z64 / math.sqrt(2)) + z64 * np.exp(-z64 ** 2 / 2) / math.sqrt(2 * math.pi), z64 ** 2),
        "gelu_tanh": (z64 * sig(u2), sig(u2) + z64 * sig(u2) * sig(-u2) * 2 * c * (1 + 3 * 0.044715 * z64 ** 2), np.abs(u2) * 3),
        "silu": (z64 * sig(z64), sig(z64) * (1 + z64 * sig(-z64)), np.abs(z64)),
    }[act]
    bar = 2 * (16 + 2 * grow) * E
    got = to64(out)
    assert (got == got[:, :1]).all()
    assert (np.abs(got[:, 0] / value - 1) <= bar).all(), float((np.abs(got[:, 0] / value - 1) / bar).max())
    # the slope, as dz = slope * 1: a sum of two addends that cancel near its zero
    dx = torch.empty_like(x)
    gy = torch.zeros(m, n, device="cuda")
    gy[:, 0] = 1
    A.attnres_linear_backward(x, w, gy, dx, activation=act)
    addends = np.abs(value / z64) + np.abs(slope - value / z64)
    err = np.abs(to64(dx[:, 0]) - slope)
    assert (err <= bar * addends).all(), float((err / (bar * addends)).max())


@gpu
@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_bf16_activations_round_once(A, act):
    """Values and slopes far below zero: off by their own rounding, and the
    exponent's relative error (a few 2^-24 of it) times 4, in fp32."""
    z = torch.linspace(-9, 9, 1024, device="cuda").bfloat16()
    x, w = torch.zeros(1024, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(64, 64, device="cuda", dtype=torch.bfloat16)
    x[:, 0], w[:, 0] = z, 1
    out, dx = torch.empty(1024, 64, device="cuda", dtype=torch.bfloat16), torch.empty_like(x)
    gy = torch.zeros_like(out)
    gy[:, 0] = 1
    A.attnres_linear(x, w, out, activation=act)
    A.attnres_linear_backward(x, w, gy, dx, activation=act)
    z64 = to64(z)
    c = math.sqrt(2 / math.pi)
    v = 2 * c * (z64 + 0.044715 * z64 ** 3) if act == "gelu_tanh" else z64
    dv = 2 * c * (1 + 3 * 0.044715 * z64 ** 2) if act == "gelu_tanh" else np.ones_like(z64)
    s, rest = 1 / (1 + np.exp(-v)), 1 / (1 + np.exp(v))
    fp32 = (16 + 4 * np.abs(v)) * 2 * E
    value, slope = z64 * s, s + z64 * s * rest * dv
    assert (np.abs(to64(out[:, 0]) - value) <= (UB + fp32) * np.abs(value) + 2.0 ** -129).all()
    # (1 - s is off by 2^-22 where it is small, times z dv, at most 80)
    bound = UB * np.abs(slope) + fp32 * (s + np.abs(z64 * s * rest * dv)) + s * np.abs(z64 * dv) * 2.0 ** -21
    assert (np.abs(to64(dx[:, 0]) - slope) <= bound + 2.0 ** -129).all()


@gpu
@pytest.mark.parametrize("dt,T,D", [(torch.bfloat16, 100, 128), (torch.bfloat16, 400, 64), (torch.bfloat16, 6000, 128), (torch.bfloat16, 300, 96),
                                    (torch.float32, 100, 40), (torch.float32, 6000, 24)])
@pytest.mark.parametrize("sign", [1, -1])
def test_an_infinite_initial_state_stays_infinite(A, dt, T, D, sign):
    """One infinite entry (d, c): outputs of channel c are infinities of q_d's
    sign, all others as without it; the final state keeps it."""
    H, d, c = 2, 5, 9
    q, k, v = (_randn(20 + i, T, H, D, dtype=dt) for i in range(3))
    decay, s0 = -torch.tensor([0.01, 0.0], device="cuda"), _randn(24, 1, H, D, D)
    runs = []
    for bad in (False, True):
        if bad:
            s0[0, :, d, c] = sign * float("inf")
        out, fin = torch.empty_like(v), torch.empty_like(s0)
        A.attnres_linear_attention(q, k, v, decay, out, initial_state=s0, final_state=fin)
        runs.append((out, fin))
    (a, fa), (b, fb) = runs
    keep = [i for i in range(D) if i != c]
    assert torch.equal(a[..., keep], b[..., keep]) and torch.equal(fa[..., keep], fb[..., keep])
    assert (b[..., c] == q[..., d].sign() * sign * float("inf")).all()
    assert (fb[0, :, d, c] == sign * float("inf")).all()
