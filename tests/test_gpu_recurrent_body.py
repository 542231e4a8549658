"""The operators together, as they are used: a stack whose body is layer norm,
projection, gated recurrence and projection (prompts, decoding, captured
graphs, rows that become padding), and a training step of such a layer whose
gradients are clipped."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from oracle import body_oracle as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def to64(t):
    return t.detach().double().cpu().numpy()


def _weights(L, d, C, dt, seed):
    from depth_wise_attention_block_gb300.bodies import GatedRecurrenceWeights
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)
    return [GatedRecurrenceWeights(w_in=normal(3 * C, d, scale=d ** -0.5, dtype=dt), w_out=normal(d, C, scale=C ** -0.5, dtype=dt),
                                   b_in=normal(3 * C, scale=0.5), b_out=normal(d, scale=0.1), norm_gain=1 + normal(d, scale=0.1),
                                   norm_bias=normal(d, scale=0.1)) for _ in range(L)]


def _setup(T, d, L, C, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h0 = torch.randn(T, d, generator=g, device="cuda").to(dt)
    W = torch.randn(L + 1, d, generator=g, device="cuda") / math.sqrt(d)
    return h0, W, _weights(L, d, C, dt, seed + 1)


def _oracle_body(w, C, cu, state):
    """v from r in fp64; `state` [n, C] is updated."""
    def body(r):
        n = B.layer_norm(r, to64(w.norm_gain), to64(w.norm_bias), 1e-5)
        xfg = B.linear(n, to64(w.w_in), to64(w.b_in))
        out, state[:], _ = B.gated_recurrence(xfg[:, :C], xfg[:, C:2 * C], xfg[:, 2 * C:], cu, state.copy())
        return B.linear(np.nan_to_num(out), to64(w.w_out), to64(w.b_out))
    return body


@pytest.mark.parametrize("C", [96, 37])
def test_stack_with_a_gated_recurrence_body(A, C):
    """fp32 stack, a ragged prompt and then three tokens per sequence, against
    the fp64 stack.  Every value passes a few thousand fp32 operations of at
    most 2^-23 per layer, and a layer's relative error may grow a few times on
    the way through the next (norms, softmax): 1e-4 of the row's largest value
    covers seven layers."""
    from depth_wise_attention_block_gb300.bodies import GatedRecurrenceBody
    from depth_wise_attention_block_gb300.stack import StackForward
    L, Bs, d = 7, 3, 200
    lens = [5, 130, 1, 24]
    n, T = len(lens), sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    h0, W, ws = _setup(T, d, L, C, torch.float32, 3)
    states = torch.zeros(L, n, C, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    body = GatedRecurrenceBody(ws, T, states, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), dev_err=err)
    fwd = StackForward(h0, W, None, None, L, Bs, body=body, dev_err=err)
    r = fwd.run().clone()
    st64 = np.zeros((L, n, C))

    def oracle(h, cu64):
        bodies = [_oracle_body(ws[l], C, cu64, st64[l]) for l in range(L)]
        return O.block_stack_forward(to64(h), to64(W), lambda l, x: bodies[l - 1](x), L, Bs).r[-1]

    def close(got, want):
        assert np.abs(to64(got) - want).max(axis=1).max() <= 1e-4 * np.abs(want).max()
    close(r, oracle(h0, cu))
    assert np.abs(to64(states) - st64).max() <= 1e-4 * np.abs(st64).max()

    # decoding: one token of each sequence, in the slots' order 2, 0, 3, 1 and a padding row
    slots = torch.tensor([2, 0, -1, 3, 1], dtype=torch.int32, device="cuda")
    live = [0, 1, 3, 4]
    order = slots[live].long().cpu().numpy()
    hd = torch.zeros(5, d, device="cuda")
    dec = GatedRecurrenceBody(ws, 5, states, decode=True, slots=slots, dev_err=err)
    step = StackForward(hd, W, None, None, L, Bs, body=dec, dev_err=err)
    for t in range(3):
        hd.normal_(generator=torch.Generator(device="cuda").manual_seed(50 + t))
        got = step.run()[live]
        st64[:] = st64[:, order]
        want = oracle(hd[live], np.arange(5))
        st64[:] = st64[:, np.argsort(order)]
        close(got, want)
    assert np.abs(to64(states) - st64).max() <= 1e-4 * np.abs(st64).max()
    assert int(err.item()) == 0


@pytest.mark.parametrize("schedule", ["single", "hybrid"])
@pytest.mark.parametrize("decode", [False, True])
def test_captured_body_gives_the_same_bits(A, schedule, decode):
    """bf16: recording advances no state, and replays equal the eager forward."""
    from depth_wise_attention_block_gb300.bodies import GatedRecurrenceBody
    from depth_wise_attention_block_gb300.stack import StackForward
    L, Bs, d, C = 6, 2, 512, 320
    T = 9 if decode else 300
    h0, W, ws = _setup(T, d, L, C, torch.bfloat16, 8)
    n = T if decode else 2
    start = torch.randn(L, n, C, device="cuda")
    states = start.clone()
    kw = dict(decode=True) if decode else dict(cu_seqlens=torch.tensor([0, 120, 300], dtype=torch.int32, device="cuda"))
    body = GatedRecurrenceBody(ws, T, states, **kw)
    fwd = StackForward(h0, W, None, None, L, Bs, body=body, schedule=schedule, two_phase_from=2, keep_weights=False)
    eager = fwd.run().clone()
    eager_states = states.clone()
    states.copy_(start)
    fwd.capture()
    assert torch.equal(states, start)
    for _ in range(2):
        states.copy_(start)
        assert torch.equal(fwd.run(), eager) and torch.equal(states, eager_states)
    assert torch.isfinite(eager).all()


def test_rows_that_become_padding_give_the_bias(A):
    from depth_wise_attention_block_gb300.bodies import GatedRecurrenceBody
    h0, _, ws = _setup(6, 64, 2, 40, torch.float32, 5)
    slots = torch.tensor([0, 1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    dec = GatedRecurrenceBody(ws, 6, torch.zeros(2, 6, 40, device="cuda"), decode=True, slots=slots)
    F = torch.empty_like(h0)
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    pre = GatedRecurrenceBody(ws, 6, torch.zeros(2, 1, 40, device="cuda"), cu_seqlens=cu)
    for body, pad in ((dec, lambda: slots[2:4].fill_(-1)), (pre, lambda: cu.copy_(torch.tensor([0, 2], dtype=torch.int32)))):
        body.issue(1, h0, F)
        body.issue(2, h0, F)
        assert not torch.allclose(F[2], ws[1].b_out)
        pad()
        body.issue(1, h0, F)
        assert torch.allclose(F[2], ws[0].b_out) and torch.allclose(F[3], ws[0].b_out) and not torch.allclose(F[1], ws[0].b_out)


def test_body_refusals(A):
    from depth_wise_attention_block_gb300.bodies import GatedRecurrenceBody
    _, _, ws = _setup(4, 64, 2, 16, torch.float32, 1)
    st = torch.zeros(2, 1, 16, device="cuda")
    with pytest.raises(ValueError, match="states"):
        GatedRecurrenceBody(ws, 4, st[:1])
    with pytest.raises(ValueError, match="states"):
        GatedRecurrenceBody(ws, 4, st[:, :, :8])
    with pytest.raises(ValueError, match="decoding"):
        GatedRecurrenceBody(ws, 4, st, slots=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="prompts"):
        GatedRecurrenceBody(ws, 4, st, decode=True, cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- training --

def _layer(f, H, p, cu):
    """aggregate -> norm -> projection -> recurrence -> projection with residual; f: the module of operations."""
    r = f.aggregate(H, p["w"])
    C = p["w_out"].shape[1]
    xfg = f.linear(f.layer_norm(r, p["gain"], p["bias"]), p["w_in"], p["b_in"])
    h, s = f.gated_recurrence(xfg[:, :C], xfg[:, C:2 * C], xfg[:, 2 * C:], cu, p["s0"])
    return f.linear(h, p["w_out"], p["b_out"], residual=r), s


class _Plain:
    """The same operations in torch, for float64."""

    @staticmethod
    def aggregate(H, w):
        z = (H * w).sum(-1) / torch.sqrt(H.square().mean(-1) + 1e-5)
        return (torch.softmax(z, 0)[..., None] * H).sum(0)

    @staticmethod
    def layer_norm(x, gain, bias):
        z = x - x.mean(-1, keepdim=True)
        return z / torch.sqrt(z.square().mean(-1, keepdim=True) + 1e-5) * gain + bias

    @staticmethod
    def linear(x, w, b, residual=None):
        z = x @ w.T + b
        return z if residual is None else z + residual

    @staticmethod
    def gated_recurrence(x, f, g, cu, s0):
        rows, ends = [], []
        for n in range(len(cu) - 1):
            h = s0[n]
            for t in range(int(cu[n]), int(cu[n + 1])):
                h = torch.sigmoid(f[t]) * h + torch.sigmoid(-f[t]) * x[t]
                rows.append(h)
            ends.append(h)
        return torch.stack(rows) * g * torch.sigmoid(g), torch.stack(ends)


def _leaves(dt, seed, T=150, d=128, C=72, S=3):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype).requires_grad_()
    return dict(H=normal(S, T, d, dtype=dt), w=normal(d, scale=d ** -0.5), gain=normal(d), bias=normal(d, scale=0.1),
                w_in=normal(3 * C, d, scale=d ** -0.5, dtype=dt), b_in=normal(3 * C, scale=0.5), w_out=normal(d, C, scale=C ** -0.5, dtype=dt),
                b_out=normal(d, scale=0.1), s0=normal(2, C))


def _run(f, leaves, cu, gy, gs):
    y, s = _layer(f, leaves["H"], leaves, cu)
    return y, s, torch.autograd.grad([y, s], list(leaves.values()), [gy.to(y.dtype), gs.to(s.dtype)])


@pytest.mark.parametrize("dt,bar", [(torch.float32, 2e-5), (torch.bfloat16, 4e-2)])
def test_training_graph_gradients_and_their_clipping(A, dt, bar):
    """Every leaf's gradient through the whole layer against float64 autograd
    of the plain operations, in the 2-norm: fp32 within 2e-5 (some 200
    operations deep at 2^-23); bf16 within ten roundings of 2^-8 on each of
    the paths a gradient takes.  Then the step's end: the gradients clipped to
    half their norm."""
    from depth_wise_attention_block_gb300 import autograd as F
    leaves = _leaves(dt, 4)
    cu = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    gy, gs = torch.randn(150, 128, generator=g, device="cuda").to(dt), torch.randn(2, 72, generator=g, device="cuda")
    y, s, grads = _run(F, leaves, cu, gy, gs)
    ref = {k: v.detach().double().requires_grad_() for k, v in leaves.items()}
    ry, rs, rgrads = _run(_Plain, ref, cu, gy.double(), gs.double())
    for name, got, want in [("y", y, ry), ("s", s, rs)] + [(n, a, b) for n, a, b in zip(leaves, grads, rgrads)]:
        rel = float((got.detach().double() - want.detach()).norm() / want.detach().norm())
        assert torch.isfinite(got).all() and rel <= bar, (name, rel)
    for leaf, grad in zip(leaves.values(), grads):
        leaf.grad = grad.clone()
    total = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    norm = F.clip_grad_norm(leaves.values(), 0.5 * total)
    assert abs(float(norm) - total) <= 2e-6 * total
    for leaf, grad in zip(leaves.values(), grads):
        want = 0.5 * grad.double()
        assert ((leaf.grad.double() - want).abs() <= ((2.0 ** -8 if grad.dtype == torch.bfloat16 else 0) + 1e-5) * want.abs() + 1e-38).all()


def test_training_graph_gradients_are_the_differences(A):
    """fp32 gradients against central differences of the float64 loss along
    random directions (whose rounding is 1e-16 / 1e-6 of the loss)."""
    from depth_wise_attention_block_gb300 import autograd as F
    leaves = _leaves(torch.float32, 5)
    cu = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    gy, gs = torch.randn(150, 128, generator=g, device="cuda"), torch.randn(2, 72, generator=g, device="cuda")
    _, _, grads = _run(F, leaves, cu, gy, gs)

    def loss(ls):
        y, s = _layer(_Plain, ls["H"], ls, cu)
        return float((y * gy).sum() + (s * gs).sum())
    base = {k: v.detach().double() for k, v in leaves.items()}
    for (name, v), grad in zip(base.items(), grads):
        u = torch.randn(v.shape, generator=g, device="cuda").double()
        h = 1e-6
        want = (loss({**base, name: v + h * u}) - loss({**base, name: v - h * u})) / (2 * h)
        got = float((grad.double() * u).sum())
        assert abs(got - want) <= 2e-5 * float(grad.double().norm() * u.norm()), (name, got, want)


def test_a_training_step_can_be_captured(A):
    """Forward, backward and clipping replayed on new inputs give the eager bits."""
    from depth_wise_attention_block_gb300 import autograd as F
    leaves = _leaves(torch.bfloat16, 6)
    cu = torch.tensor([0, 70, 150], dtype=torch.int32, device="cuda")
    gy, gs = torch.randn(150, 128, device="cuda").bfloat16(), torch.randn(2, 72, device="cuda")

    def step():
        _, _, grads = _run(F, leaves, cu, gy, gs)
        norm = torch.empty(1, device="cuda")
        A.attnres_grad_clip(grads, 1.0, norm)
        return [*grads, norm]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    gy.normal_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in held]
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


def test_stack_backward_clips_its_gradients(A):
    import workloads
    from depth_wise_attention_block_gb300.stack import StackBackward, StackForward
    stk = workloads.stack(T=8, d=256, num_layers=4, block_size=2, seed=12, device=torch.device("cuda"), dtype=torch.float32)
    fwd = StackForward(stk.h0, stk.W, stk.G, stk.Sc, 4, 2, keep_weights=False)
    fwd.run()
    bwd = StackBackward(fwd)
    dh0, dW = bwd.run(torch.randn(8, 256, device="cuda"))
    other = torch.randn(77, device="cuda")
    dh, dw, o = dh0.clone(), dW.clone(), other.clone()
    want = math.sqrt(float(dw.double().square().sum() + o.double().square().sum()))
    norm = bwd.clip(0.25 * want, [other])
    assert abs(float(norm) - want) <= 2e-6 * want
    assert torch.equal(dh0, dh) and torch.allclose(dW, 0.25 * dw, rtol=1e-5) and torch.allclose(other, 0.25 * o, rtol=1e-5)
