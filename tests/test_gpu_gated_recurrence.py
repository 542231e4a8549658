"""attnres_gated_recurrence, its backward and its step on the GPU against
their fp64 statements.

Tolerances, derived from the arithmetic before any run.  e = 2^-23 bounds one
fp32 operation, u is half a rounding step of the stored type (bf16 2^-8, fp32
2^-24).  a and 1 - a are each off by (|f| + 16) e of themselves: the exponent's
argument f log2 e by |f| e, an exponential, a sum, a reciprocal and a product
by a few e.  With c the recurrence over absolute values, c_t = a c_{t-1} +
(1 - a) |x|, every step adds (|f| + 16) e c_t to an error that decays as the
state does: E_t = a E_{t-1} + (|f| + 16) e c_t (the products of gates that
carry a state over a span are off by the sum of their factors' errors, which
these terms count factor by factor).  sigma(g) and 1 - sigma(g): (|g| + 16) e.
Gates below -83 count as -83, and fp32 has a smallest number: + 1e-34 of the
largest value that such a gate multiplies."""
import numpy as np
import pytest
import torch

from oracle import body_oracle as B

pytestmark = pytest.mark.gpu
E = 2.0 ** -23
TINY = 1e-33
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def to64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _randn(seed, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def _close(got, want, bound, what):
    got = to64(got)
    live = ~np.isnan(want)
    assert np.isfinite(got[live]).all(), what
    err = np.abs(got - want)[live]
    bound = np.broadcast_to(bound, want.shape)[live] + TINY
    worst = (err / bound).max() if err.size else 0.0
    assert (err <= bound).all(), f"{what}: worst {worst:.3g} x bound"


def _inputs(T, C, n, dt, gate, seed, wide=0, fshift=2.0):
    """x, f, g, dy: slices of wider buffers, `wide` elements apart."""
    def rows(k, **kw):
        return _randn(seed + k, T, C + 2 * wide, dtype=dt, **kw)[:, wide:wide + C]
    return (rows(0), rows(1, scale=2.0, shift=fshift), rows(2) if gate else None, rows(3), _randn(seed + 4, n, C), _randn(seed + 5, n, C))


def _bounds(x, f, g, cu, s0, dy, ds1):
    """(E of h, of states before; E of dh, c of dh; c) by the recurrences of the module's text."""
    a, rest = B.sigmoid(f), B.sigmoid(-f)
    T, C = x.shape
    n = len(cu) - 1
    eh, ebefore, c, cbefore = (np.zeros((T, C)) for _ in range(4))
    ed, cd = np.zeros((T, C)), np.zeros((T, C))
    efin, ed0 = np.zeros((n, C)), np.zeros((n, C))
    kap = (np.abs(f) + 16) * E
    s = np.abs(B.silu(g)) * np.ones((T, C))
    kg = 0.0 if g is None else (np.abs(g) + 16) * E
    for i in range(n):
        ct, et = (np.zeros(C) if s0 is None else np.abs(s0[i])), np.zeros(C)
        for t in range(cu[i], cu[i + 1]):
            ebefore[t], cbefore[t] = et, ct
            ct = a[t] * ct + rest[t] * np.abs(x[t])
            et = a[t] * et + kap[t] * ct
            eh[t], c[t] = et, ct
        efin[i] = et
        ct, et = (np.zeros(C) if ds1 is None else np.abs(ds1[i])), np.zeros(C)
        for t in range(cu[i + 1] - 1, cu[i] - 1, -1):
            if dy is None:
                break
            ct = ct + np.abs(dy[t]) * s[t]
            et = et + (kg if g is None else kg[t]) * np.abs(dy[t]) * s[t] + 2 * E * ct
            ed[t], cd[t] = et, ct
            et = a[t] * et + kap[t] * a[t] * ct
            ct = a[t] * ct
        ed0[i] = et
    return eh, ebefore, c, efin, ed, cd, ed0


def _run(A, x, f, g, cu, s0, dy, ds1, dt, what, backward=True):
    T, C = x.shape
    n = 1 if cu is None else len(cu) - 1
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.full((T, C), float("nan"), dtype=dt, device="cuda")
    fin = torch.full((n, C), float("nan"), device="cuda")
    chunk = torch.full((-(-T // 64), C), float("nan"), device="cuda")
    A.attnres_gated_recurrence(x, f, out, gate=g, cu_seqlens=cut, initial_state=s0, final_state=fin, chunk_states=chunk)
    cu = [0, T] if cu is None else [min(max(c, 0), T) for c in cu]
    X, F, G, S0, DY, DS1 = (to64(t) for t in (x, f, g, s0, dy, ds1))
    want, wfin, before = B.gated_recurrence(X, F, G, cu, S0)
    eh, eb, c, efin, ed, cd, ed0 = _bounds(X, F, G, cu, S0, DY if backward else None, DS1)
    gs = 1.0 if G is None else np.abs(B.silu(G))
    ge = 0.0 if G is None else (np.abs(G) + 16) * E
    _close(out, want, gs * eh + (ge + 2 * E + U[dt]) * np.abs(want), (what, "out"))
    live = np.zeros(T, bool)
    live[cu[0]:cu[-1]] = True
    assert np.isnan(to64(out)[~live]).all(), "rows outside every sequence"
    _close(fin, wfin, efin, (what, "final"))
    if not backward:
        return out, fin
    # gradients side by side in one buffer, as a projection's rows are
    buf = torch.full((T, 3 * C + 4), 7.0, dtype=dt, device="cuda")
    gx, gf, gg = buf[:, :C], buf[:, C:2 * C], buf[:, 2 * C:3 * C] if g is not None else None
    ds0 = torch.full((n, C), float("nan"), device="cuda")
    A.attnres_gated_recurrence_backward(x, f, chunk, dy, gx, gf, gg, gate=g, cu_seqlens=cut, initial_state=s0, grad_final_state=ds1,
                                        grad_initial_state=ds0)
    dx, df, dg, wds0 = B.gated_recurrence_backward(X, F, G, cu, S0, DY, DS1)
    a, rest, kap = B.sigmoid(F), B.sigmoid(-F), (np.abs(F) + 16) * E
    _close(gx[live], dx[live], (rest * (ed + (kap + E) * cd) + U[dt] * np.abs(dx))[live], (what, "grad_x"))
    ar, gap = a * rest, np.abs(before - X)
    err = ar * (gap * (ed + (2 * kap + 4 * E) * cd) + cd * (eb + E * (np.abs(before) + np.abs(X)))) + U[dt] * np.abs(df)
    _close(gf[live], df[live], err[live], (what, "grad_forget"))
    if g is not None:
        sg = B.sigmoid(G)
        slope_err = (np.abs(G) + 16) * E * sg * (1 + 2 * np.abs(G))
        err = np.abs(DY) * ((eh + 2 * E * c) * np.abs(B.silu_slope(G)) + c * slope_err) + U[dt] * np.abs(dg)
        _close(gg[live], dg[live], err[live], (what, "grad_gate"))
    else:
        assert (buf[:, 2 * C:] == 7).all()
    assert (buf[~torch.tensor(live)] == 7).all() and (buf[:, 3 * C:] == 7).all()
    _close(ds0, wds0, ed0, (what, "grad_initial"))
    return out, fin, chunk, buf, ds0


# one token, lengths around the chunk of 64, channels of less than a vector and
# a lane, odd, more than one slab of channels; enough rows for several groups
SIZES = [(1, 1), (1, 64), (2, 3), (5, 8), (63, 7), (64, 64), (65, 66), (127, 33), (128, 130), (200, 1), (300, 200), (513, 40), (1000, 65),
         (700, 517), (2111, 24), (4100, 16), (1300, 1000)]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,C", SIZES)
def test_one_sequence(A, T, C, dt):
    for seed, (gate, state, wide) in enumerate([(True, True, 0), (False, False, 0), (True, False, 16), (False, True, 3)]):
        x, f, g, dy, s0, ds1 = _inputs(T, C, 1, dt, gate, 10 * seed, wide)
        _run(A, x, f, g, None, s0 if state else None, dy, ds1 if state else None, dt, (gate, state, wide))


# empty sequences at the start, inside, many in a row and at the end; rows ahead
# of the first and behind the last; lengths of one; ends on a chunk's border;
# offsets outside 0..T
CUTS = [(100, [0, 0, 1, 2, 40, 40, 100, 100]), (130, [5, 64, 64, 128]), (300, [0] + [100] * 40 + [300]), (257, [3, 4, 5, 6, 7, 250]),
        (64, list(range(0, 65))), (500, [0, 64, 128, 192, 256, 500]), (90, [-7, 30, 200]), (40, [40, 40, 40]), (50, [0, 0]),
        (1000, [0, 300, 301, 999, 1000]), (3000, [1, 700, 700, 1500, 2990])]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,cu", CUTS, ids=lambda v: str(v) if isinstance(v, int) else str(len(v)))
def test_ragged(A, T, cu, dt):
    n = len(cu) - 1
    for seed, (C, gate, state, wide) in enumerate([(72, True, True, 0), (72, False, False, 0), (35, True, True, 1)]):
        x, f, g, dy, s0, ds1 = _inputs(T, C, n, dt, gate, 20 + seed, wide)
        _run(A, x, f, g, cu, s0 if state else None, dy, ds1 if state else None, dt, (C, gate, state))


def test_many_short_sequences(A):
    r = np.random.default_rng(0)
    lens = r.integers(0, 4, size=900)
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    x, f, g, dy, s0, ds1 = _inputs(cu[-1] + 5, 40, 900, torch.float32, True, 3)
    _run(A, x, f, g, cu, s0, dy, ds1, torch.float32, "short")


@pytest.mark.parametrize("dt", DTYPES)
def test_memories_from_none_to_hundreds_of_tokens(A, dt):
    T, C = 1500, 64
    x, _, g, dy, s0, ds1 = _inputs(T, C, 2, dt, True, 5)
    f = torch.linspace(-100, 9, C, device="cuda").expand(T, C).contiguous().to(dt)
    _run(A, x, f, g, [0, 700, T], s0, dy, ds1, dt, "gates")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,C,cu", [(1, 1, None), (15, 7, None), (200, 63, None), (333, 65, [0, 5, 130, 333]), (70, 130, [3, 40, 60]),
                                    (64, 8, [0, 64]), (1100, 300, [0, 1100]),
                                    (130, 128, None), (500, 72, [2, 130, 131, 488])])
def test_rows_on_vectors_and_off_them(A, T, C, cu, dt):
    """Rows of 16-byte vectors (channels that fill them or not) and the same
    rows one element off give the same bits, and nothing beside them is written."""
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    n = 1 if cu is None else len(cu) - 1
    x, f, g, dy, s0, ds1 = _inputs(T, C, n, dt, True, 11)
    pitch = -(-C // 8) * 8 + 8
    results = []
    for off in (0, 1):
        def rows(t):
            buf = torch.full((T, pitch), 7.0, dtype=dt, device="cuda")
            buf[:, off:off + C] = t
            return buf, buf[:, off:off + C]
        ins = [rows(t)[1] for t in (x, f, g, dy)]
        outs = [rows(7.0) for _ in range(4)]
        out, dx, df, dg = (view for _, view in outs)
        fin, ds0 = torch.full((n, C), 7.0, device="cuda"), torch.full((n, C), 7.0, device="cuda")
        chunk = torch.empty(-(-T // 64), C, device="cuda")
        A.attnres_gated_recurrence(ins[0], ins[1], out, gate=ins[2], cu_seqlens=cut, initial_state=s0, final_state=fin, chunk_states=chunk)
        A.attnres_gated_recurrence_backward(ins[0], ins[1], chunk, ins[3], dx, df, dg, gate=ins[2], cu_seqlens=cut, initial_state=s0,
                                            grad_final_state=ds1, grad_initial_state=ds0)
        live = torch.zeros(T, pitch, dtype=torch.bool, device="cuda")
        live[(cu or [0])[0]:(cu or [T])[-1], off:off + C] = True
        assert all((buf[~live] == 7).all() for buf, _ in outs)
        results.append([out.clone(), dx.clone(), df.clone(), dg.clone(), fin, ds0])
    for one, other in zip(*results):
        assert torch.equal(one, other)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("C", [48, 35])
def test_states_in_place_and_the_same_bits(A, C, dt):
    cu = [0, 130, 130, 131, 600]
    x, f, g, dy, s0, ds1 = _inputs(600, C, 4, dt, True, 7)
    out, fin, chunk, buf, ds0 = _run(A, x, f, g, cu, s0, dy, ds1, dt, "apart")
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st, out2 = s0.clone(), torch.empty_like(out)
    A.attnres_gated_recurrence(x, f, out2, gate=g, cu_seqlens=cut, initial_state=st, final_state=st)
    assert torch.equal(st, fin) and torch.equal(out, out2)
    d, grads = ds1.clone(), torch.empty(3, 600, C, dtype=dt, device="cuda")
    A.attnres_gated_recurrence_backward(x, f, chunk, dy, *grads, gate=g, cu_seqlens=cut, initial_state=s0, grad_final_state=d,
                                        grad_initial_state=d)
    assert torch.equal(d, ds0)
    for i in range(3):
        assert torch.equal(grads[i], buf[:, i * C:(i + 1) * C])
    # gradients one at a time
    for i in range(4):
        one = [torch.empty(600, C, dtype=dt, device="cuda") if i == j else None for j in range(3)]
        d0 = torch.empty_like(ds0) if i == 3 else None
        A.attnres_gated_recurrence_backward(x, f, chunk, dy, *one, gate=g, cu_seqlens=cut, initial_state=s0, grad_final_state=ds1,
                                            grad_initial_state=d0)
        assert torch.equal(d0, ds0) if i == 3 else torch.equal(one[i], grads[i])


@pytest.mark.parametrize("dt", DTYPES)
def test_infinities_stay_in_their_channel_and_sequence(A, dt):
    cu = [0, 70, 200, 330]
    x, f, g, dy, s0, ds1 = _inputs(330, 70, 3, dt, True, 9)
    out, fin, chunk, buf, ds0 = _run(A, x, f, g, cu, s0, dy, ds1, dt, "clean")
    x2, f2, dy2, s2, d2 = x.clone(), f.clone(), dy.clone(), s0.clone(), ds1.clone()
    x2[100, 3], f2[90, 8], x2[120, 20] = float("inf"), float("nan"), float("nan")
    s2[1, 30], dy2[110, 40], d2[1, 50] = float("inf"), float("inf"), float("nan")
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, fn, ch = torch.empty_like(out), torch.empty_like(fin), torch.empty_like(chunk)
    A.attnres_gated_recurrence(x2, f2, o, gate=g, cu_seqlens=cut, initial_state=s2, final_state=fn, chunk_states=ch)
    bad = [3, 8, 20, 30]
    good = [c for c in range(70) if c not in bad]
    rows = torch.cat([torch.arange(0, 70), torch.arange(200, 330)])
    assert torch.equal(o[rows], out[rows]) and torch.equal(o[:, good], out[:, good])
    assert torch.equal(fn[[0, 2]], fin[[0, 2]]) and torch.equal(fn[:, good], fin[:, good])
    for c, t in ((3, 100), (8, 90), (20, 120), (30, 70)):
        assert not torch.isfinite(o[t:200, c]).any() and torch.equal(o[70:t, c], out[70:t, c]) and not torch.isfinite(fn[1, c])
    grads, d0 = torch.full((3, 330, 70), 7.0, dtype=dt, device="cuda"), torch.empty_like(ds0)
    A.attnres_gated_recurrence_backward(x2, f2, ch, dy2, *grads, gate=g, cu_seqlens=cut, initial_state=s2, grad_final_state=d2,
                                        grad_initial_state=d0)
    good = [c for c in good if c not in (40, 50)]
    for i in range(3):
        want = buf[:, i * 70:(i + 1) * 70]
        assert torch.equal(grads[i][rows], want[rows]) and torch.equal(grads[i][:, good], want[:, good])
    assert torch.equal(d0[[0, 2]], ds0[[0, 2]]) and torch.equal(d0[:, good], ds0[:, good])
    assert not torch.isfinite(grads[0][70:111, 40]).any() and not torch.isfinite(grads[0][70:200, 50]).any()


def test_gates_of_infinity(A):
    """A forget gate of -inf starts again from the input, one of +inf keeps the state."""
    x = _randn(1, 200, 40)
    f = torch.full_like(x, 1.0)
    f[50], f[100] = float("-inf"), float("inf")
    out = torch.empty_like(x)
    A.attnres_gated_recurrence(x, f, out)
    assert torch.allclose(out[50], x[50], rtol=1e-6, atol=0) and torch.equal(out[100], out[99]) and torch.isfinite(out).all()


def test_no_rows(A):
    e = torch.empty(0, 24, device="cuda")
    s0, fin = _randn(1, 3, 24), torch.empty(3, 24, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    A.attnres_gated_recurrence(e, e, e, cu_seqlens=cu, initial_state=s0, final_state=fin)
    assert torch.equal(fin, s0)
    A.attnres_gated_recurrence(e, e, e, final_state=fin[:1])
    assert not fin[0].any()
    ds0 = torch.empty_like(fin)
    A.attnres_gated_recurrence_backward(e, e, e, e, None, None, cu_seqlens=cu, grad_final_state=s0, grad_initial_state=ds0)
    assert torch.equal(ds0, s0)


# ---------------------------------------------------------------- decoding --

@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("B_,C", [(1, 1), (1, 7168), (3, 8), (5, 33), (64, 200), (130, 66), (9, 1030)])
def test_step(A, B_, C, dt):
    r = np.random.default_rng(B_)
    for seed, (gate, wide, named) in enumerate([(True, 0, True), (False, 8, True), (True, 3, False)]):
        ns = B_ + 3
        x, f, g, _, _, _ = _inputs(B_, C, 1, dt, gate, 30 + seed, wide)
        state = _randn(40 + seed, ns, C)
        slots = r.permutation(ns)[:B_]
        if B_ > 4:  # padding rows and a slot named three times
            slots[1], slots[2] = -1, ns + 5
            slots[B_ - 1] = slots[3] = slots[0]
        if not named:
            slots = np.arange(B_)
        out = torch.full((B_, C), float("nan"), dtype=dt, device="cuda")
        S = to64(state)
        want, wst = B.gated_recurrence_step(to64(x), to64(f), to64(g), S, slots)
        A.attnres_gated_recurrence_step(x, f, state, out, gate=g, slots=torch.tensor(slots, dtype=torch.int32, device="cuda") if named else None)
        # at most three steps of one slot: three times the injected error of the largest value there
        F, X = np.abs(to64(f)), np.abs(to64(x))
        c = np.maximum(np.abs(S).max(0), X.max(0))
        es = 3 * (F.max(0) + 16) * E * c
        _close(state, wst, es, "state")
        G = to64(g)
        gs, ge = (1.0, 0.0) if G is None else (np.abs(B.silu(G)), (np.abs(G) + 16) * E)
        _close(out, want, gs * es + (ge + 2 * E + U[dt]) * np.abs(want), "out")
        pad = np.isnan(want).all(1)
        assert np.isnan(to64(out)[pad]).all()


def test_a_prompt_and_its_steps_agree(A):
    """A prompt's states go on token by token: the same recurrence on the bars of one."""
    T, C = 90, 136
    x, f, g, _, s0, _ = _inputs(T, C, 1, torch.float32, True, 50)
    whole, fin = torch.empty_like(x), torch.empty(1, C, device="cuda")
    A.attnres_gated_recurrence(x, f, whole, gate=g, initial_state=s0, final_state=fin)
    st, out = torch.zeros(4, C, device="cuda"), torch.empty_like(x)
    A.attnres_gated_recurrence(x[:50], f[:50], out[:50], gate=g[:50], initial_state=s0, final_state=st[2:3])
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    for t in range(50, T):
        A.attnres_gated_recurrence_step(x[t:t + 1], f[t:t + 1], st, out[t:t + 1], gate=g[t:t + 1], slots=slot)
    eh, *_, = _bounds(to64(x), to64(f), to64(g), [0, T], to64(s0), None, None)
    assert (np.abs(to64(out) - to64(whole)) <= 2 * (np.abs(B.silu(to64(g))) * eh + 20 * E * np.abs(to64(whole))) + TINY).all()
    assert not st[[0, 1, 3]].any()


# ------------------------------------------------------ streams and graphs --

def test_streams_and_graphs(A):
    dt = torch.bfloat16
    x, f, g, dy, s0, ds1 = _inputs(3000, 264, 3, dt, True, 60)
    cu = torch.tensor([0, 900, 910, 3000], dtype=torch.int32, device="cuda")
    out, fin, chunk = torch.empty_like(x), torch.empty_like(s0), torch.empty(47, 264, device="cuda")
    grads, ds0 = torch.empty(3, 3000, 264, dtype=dt, device="cuda"), torch.empty_like(s0)

    def call(stream=None):
        A.attnres_gated_recurrence(x, f, out, gate=g, cu_seqlens=cu, initial_state=s0, final_state=fin, chunk_states=chunk, stream=stream)
        A.attnres_gated_recurrence_backward(x, f, chunk, dy, *grads, gate=g, cu_seqlens=cu, initial_state=s0, grad_final_state=ds1,
                                            grad_initial_state=ds0, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in (out, fin, grads, ds0)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in (out, fin, grads, ds0, chunk):
        t.zero_()
    for _ in range(2):
        graph.replay()
    for t, v in zip((out, fin, grads, ds0), want):
        assert torch.equal(t, v)
    # offsets written over between replays
    cu.copy_(torch.tensor([0, 10, 2000, 2500], dtype=torch.int32))
    graph.replay()
    got = [t.clone() for t in (out, fin, grads, ds0)]
    call()
    for t, v in zip((out, fin, grads, ds0), got):
        assert torch.equal(t, v)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T,C", [(2000, 40), (700, 300)])
def test_waits_that_run_out(A, T, C, dt):
    """The bounded waits of a cluster's CTAs on one another, made to run out on
    a healthy GPU (attnres_debug_wait_test: the first tiles' spans are not
    sent): the call reports it, writes NaN and returns, and the same call then
    gives the same bits as before."""
    x, f, g, dy, s0, ds1 = _inputs(T, C, 1, dt, True, 80)
    out, fin, chunk = torch.empty(T, C, dtype=dt, device="cuda"), torch.empty_like(s0), torch.empty(-(-T // 64), C, device="cuda")
    grads, ds0 = torch.empty(3, T, C, dtype=dt, device="cuda"), torch.empty_like(s0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        A.attnres_gated_recurrence(x, f, out, gate=g, initial_state=s0, final_state=fin, chunk_states=chunk, dev_err=err)
        A.attnres_gated_recurrence_backward(x, f, chunk, dy, *grads, gate=g, initial_state=s0, grad_final_state=ds1,
                                            grad_initial_state=ds0, dev_err=err)
        torch.cuda.synchronize()
    call()
    assert int(err.item()) == 0
    want = [t.clone() for t in (out, fin, grads, ds0)]
    A.attnres_debug_wait_test(1_000_000, 0)
    try:
        call()
    finally:
        A.attnres_debug_wait_test(0, -1)
    assert int(err.item()) & A.ATTNRES_DEVERR_WAIT_TIMEOUT
    for t in (out, fin, grads, ds0):
        assert torch.isnan(t).all()
    err.zero_()
    call()
    assert int(err.item()) == 0
    for t, v in zip((out, fin, grads, ds0), want):
        assert torch.equal(t, v)


@pytest.mark.parametrize("dt", DTYPES)
def test_autograd(A, dt):
    from depth_wise_attention_block_gb300 import autograd as F
    cu = [2, 70, 70, 150]
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    x, f, g, dy, s0, ds1 = _inputs(160, 40, 3, dt, True, 70)
    names = ("x", "f", "g", "s0")
    for need in [(1, 1, 1, 1), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1)]:
        leaves = [t.detach().clone().requires_grad_(bool(k)) for t, k in zip((x, f, g, s0), need)]
        out, fin = F.gated_recurrence(*leaves[:3], cut, leaves[3])
        assert not out[:2].any() and not out[150:].any()
        torch.autograd.backward([out, fin], [dy, ds1])
        want = dict(zip(names, B.gated_recurrence_backward(*(to64(t) for t in (x, f, g)), cu, to64(s0), to64(dy), to64(ds1))))
        for name, leaf, k in zip(names, leaves, need):
            assert (leaf.grad is not None) == bool(k)
            if k:
                w = np.nan_to_num(want[name])
                rel = np.linalg.norm(to64(leaf.grad) - w) / np.linalg.norm(w)
                assert rel <= (U[dt] if name != "s0" else 0) + 1e-5, (name, rel)
    # without gates and states; a prompt without a gradient keeps nothing
    x1, f1 = x.detach().clone().requires_grad_(), f.detach().clone()
    out, fin = F.gated_recurrence(x1, f1)
    fin.sum().backward()
    assert torch.isfinite(x1.grad).all() and x1.grad.any()
    assert F.gated_recurrence(x, f)[0].grad_fn is None
