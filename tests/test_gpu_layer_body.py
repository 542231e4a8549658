"""The operators together, as a layer body uses them: a stack whose body is a
linear-attention layer (prompts, decoding, captured graphs, the two-phase
schedule), and the differentiable operations in one training graph."""
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


def _weights(L, d, heads, Dk, Dv, dt, seed):
    from depth_wise_attention_block_gb300.bodies import LinearAttentionWeights
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)
    return [LinearAttentionWeights(
        w_qkv=normal(heads * (2 * Dk + Dv), d, scale=d ** -0.5, dtype=dt),
        w_out=normal(d, heads * Dv, scale=0.5 * (heads * Dv) ** -0.5, dtype=dt),
        b_qkv=normal(heads * (2 * Dk + Dv), scale=0.1), b_out=normal(d, scale=0.1),
        q_gain=1 + normal(Dk, scale=0.1), k_gain=1 + normal(Dk, scale=0.1)) for _ in range(L)]


def _setup(T, d, L, heads, Dk, Dv, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h0 = torch.randn(T, d, generator=g, device="cuda").to(dt)
    W = torch.randn(L + 1, d, generator=g, device="cuda") / math.sqrt(d)
    decay = -torch.exp2(-1.0 - 4.0 * torch.arange(heads, device="cuda") / heads)
    freq = (1000.0 ** (-torch.arange(0, Dk, 2, device="cuda").double() / Dk)).float()
    return h0, W, decay, freq, _weights(L, d, heads, Dk, Dv, dt, seed + 1)


def _oracle_body(w, heads, Dk, Dv, decay, freq, pos, cu, state):
    """v from r in fp64; `state` [n, heads, Dk, Dv] is updated."""
    def body(r):
        T = r.shape[0]
        qkv = B.linear(r, to64(w.w_qkv), to64(w.b_qkv))
        q = qkv[:, :heads * Dk].reshape(T, heads, Dk)
        k = qkv[:, heads * Dk:2 * heads * Dk].reshape(T, heads, Dk)
        v = qkv[:, 2 * heads * Dk:].reshape(T, heads, Dv)
        q = B.qk_norm_rope(q, to64(w.q_gain), pos, to64(freq), False, 1e-5)
        k = B.qk_norm_rope(k, to64(w.k_gain), pos, to64(freq), False, 1e-5)
        out, state[:] = B.linear_attention(q, k, v, to64(decay), cu, state.copy(), Dk ** -0.5)
        return B.linear(out.reshape(T, -1), to64(w.w_out), to64(w.b_out))
    return body


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (40, 24)])
def test_stack_with_a_linear_attention_body(A, Dk, Dv):
    """fp32 stack, a ragged prompt and then three tokens per sequence, against
    the fp64 stack.  Every value passes a few thousand fp32 operations of at
    most 2^-23 per layer, and a layer's relative error may grow a few times on
    the way through the next (norms, softmax): 1e-4 of the row's largest value
    covers seven layers."""
    from depth_wise_attention_block_gb300.bodies import LinearAttentionBody
    from depth_wise_attention_block_gb300.stack import StackForward
    L, Bs, d, heads = 7, 3, 256, 3
    lens = [5, 130, 1, 24]
    n, T = len(lens), sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    h0, W, decay, freq, ws = _setup(T, d, L, heads, Dk, Dv, torch.float32, 3)
    states = torch.zeros(L, n, heads, Dk, Dv, device="cuda")
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    body = LinearAttentionBody(ws, T, heads, Dk, Dv, decay, states, positions=pos, inv_freq=freq,
                               cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), dev_err=err)
    fwd = StackForward(h0, W, None, None, L, Bs, body=body, dev_err=err)
    r = fwd.run().clone()
    st64 = np.zeros((L, n, heads, Dk, Dv))

    def oracle(h, pos64, cu64):
        bodies = [_oracle_body(ws[l], heads, Dk, Dv, decay, freq, pos64, cu64, st64[l]) for l in range(L)]
        return O.block_stack_forward(to64(h), to64(W), lambda l, x: bodies[l - 1](x), L, Bs).r[-1]

    def close(got, want):
        assert np.abs(to64(got) - want).max(axis=1).max() <= 1e-4 * np.abs(want).max()
    close(r, oracle(h0, to64(pos), cu))
    assert np.abs(to64(states) - st64).max() <= 1e-4 * np.abs(st64).max()

    # decoding: one token of each sequence, in the slots' order 2, 0, 3, 1 and a padding row
    slots = torch.tensor([2, 0, -1, 3, 1], dtype=torch.int32, device="cuda")
    live = [0, 1, 3, 4]
    order = slots[live].long()
    hd = torch.zeros(5, d, device="cuda")
    p = torch.tensor([lens[s] if s >= 0 else 0 for s in slots.tolist()], device="cuda")
    dec = LinearAttentionBody(ws, 5, heads, Dk, Dv, decay, states, positions=p, inv_freq=freq, decode=True, slots=slots, dev_err=err)
    step = StackForward(hd, W, None, None, L, Bs, body=dec, dev_err=err)
    for t in range(3):
        hd.normal_(generator=torch.Generator(device="cuda").manual_seed(50 + t))
        got = step.run()[live]
        st64[:] = st64[:, order.cpu().numpy()]
        want = oracle(hd[live], to64(p[live]), np.arange(5))
        back = np.argsort(order.cpu().numpy())
        st64[:] = st64[:, back]
        close(got, want)
        p += 1
    assert np.abs(to64(states) - st64).max() <= 1e-4 * np.abs(st64).max()
    assert int(err.item()) == 0


@pytest.mark.parametrize("schedule", ["single", "hybrid"])
@pytest.mark.parametrize("decode", [False, True])
def test_captured_body_gives_the_same_bits(A, schedule, decode):
    """bf16: a captured stack replayed on new rows equals the eager one."""
    from depth_wise_attention_block_gb300.bodies import LinearAttentionBody
    from depth_wise_attention_block_gb300.stack import StackForward
    L, Bs, d, heads, D = 6, 2, 512, 4, 128
    T = 9 if decode else 300
    h0, W, decay, freq, ws = _setup(T, d, L, heads, D, D, torch.bfloat16, 8)
    n = T if decode else 2
    start = torch.randn(L, n, heads, D, D, device="cuda")
    states = start.clone()
    kw = dict(decode=True) if decode else dict(cu_seqlens=torch.tensor([0, 120, 300], dtype=torch.int32, device="cuda"))
    body = LinearAttentionBody(ws, T, heads, D, D, decay, states, positions=torch.arange(T, device="cuda"), inv_freq=freq, **kw)
    fwd = StackForward(h0, W, None, None, L, Bs, body=body, schedule=schedule, two_phase_from=2, keep_weights=False)
    eager = fwd.run().clone()
    eager_states = states.clone()
    fwd.capture()
    for _ in range(2):
        states.copy_(start)
        assert torch.equal(fwd.run(), eager) and torch.equal(states, eager_states)
    assert torch.isfinite(eager).all()
    with pytest.raises(ValueError, match="stand-in"):
        fwd.bytes_moved()
    with pytest.raises(ValueError, match="stand-in"):
        fwd.launches_per_forward()


def test_body_refusals(A):
    from depth_wise_attention_block_gb300.bodies import LinearAttentionBody
    from depth_wise_attention_block_gb300.stack import StackBackward, StackForward
    h0, W, decay, freq, ws = _setup(4, 64, 2, 2, 16, 16, torch.float32, 1)
    st = torch.zeros(2, 1, 2, 16, 16, device="cuda")
    with pytest.raises(ValueError, match="states"):
        LinearAttentionBody(ws, 4, 2, 16, 16, decay, st[:1])
    with pytest.raises(ValueError, match="decoding"):
        LinearAttentionBody(ws, 4, 2, 16, 16, decay, st, slots=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="prompts"):
        LinearAttentionBody(ws, 4, 2, 16, 16, decay, st, decode=True, cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="G and Sc"):
        StackForward(h0, W, None, None, 2, 2)
    fwd = StackForward(h0, W, None, None, 2, 2, body=LinearAttentionBody(ws, 4, 2, 16, 16, decay, st))
    with pytest.raises(ValueError, match="stand-in"):
        StackBackward(fwd)


# ---------------------------------------------------------------- training --

def _layer(f, H, w, p, decay, pos, freq, heads, D, cu, s0):
    """aggregate -> projection -> norm and rotation -> attention -> projection
    with activation and residual; f: the module of operations."""
    r = f.aggregate(H, w)
    T = r.shape[0]
    qkv = f.linear(r, p["w_qkv"], p["b_qkv"])
    q, k, v = (qkv[:, i * heads * D:(i + 1) * heads * D].unflatten(1, (heads, D)) for i in range(3))
    q, k = f.qk_norm_rope(q, k, p["q_gain"], p["k_gain"], pos, freq)
    o, s = f.linear_attention(q, k, v, decay, cu, s0)
    return f.linear(o.reshape(T, heads * D), p["w_out"], p["b_out"], residual=r, activation="silu"), s


class _Plain:
    """The same operations in torch, for float64."""

    @staticmethod
    def aggregate(H, w):
        z = (H * w).sum(-1) / torch.sqrt(H.square().mean(-1) + 1e-5)
        return (torch.softmax(z, 0)[..., None] * H).sum(0)

    @staticmethod
    def linear(x, w, b, residual=None, activation="none"):
        z = x @ w.T + b
        z = z * torch.sigmoid(z) if activation == "silu" else z
        return z if residual is None else z + residual

    @staticmethod
    def qk_norm_rope(q, k, qg, kg, pos, freq):
        def one(x, g):
            y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * g
            ang = pos.double()[:, None, None] * freq.double()
            a, b = y.chunk(2, -1)
            return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
        return one(q, qg), one(k, kg)

    @staticmethod
    def linear_attention(q, k, v, g, cu, s0):
        outs, ends = [], []
        for n in range(len(cu) - 1):
            a, b = int(cu[n]), int(cu[n + 1])
            i = torch.arange(b - a, device=q.device)
            gap = (i[:, None] - i[None, :])
            D = torch.where(gap >= 0, torch.exp(g[:, None, None].double() * gap.clamp(min=0)), 0.0)
            qs, ks, vs = (t[a:b].transpose(0, 1) for t in (q, k, v))
            up = torch.exp(g[:, None, None].double() * (i[:, None] + 1))
            outs.append((((qs @ ks.transpose(1, 2) * D) @ vs + up * (qs @ s0[n])) * q.shape[2] ** -0.5).transpose(0, 1))
            down = torch.exp(g[:, None, None].double() * (b - a - 1 - i[:, None]))
            ends.append(torch.exp(g[:, None, None].double() * (b - a)) * s0[n] + (ks * down).transpose(1, 2) @ vs)
        return torch.cat(outs), torch.stack(ends)


def _leaves(dt, seed, T=200, d=128, heads=2, D=64, S=3):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype).requires_grad_()
    leaves = dict(H=normal(S, T, d, dtype=dt), w=normal(d, scale=d ** -0.5), w_qkv=normal(3 * heads * D, d, scale=d ** -0.5, dtype=dt),
                  b_qkv=normal(3 * heads * D, scale=0.1), q_gain=normal(D), k_gain=normal(D),
                  w_out=normal(d, heads * D, scale=(heads * D) ** -0.5, dtype=dt), b_out=normal(d, scale=0.1),
                  s0=normal(2, heads, D, D))
    fixed = dict(decay=-torch.tensor([0.02, 0.4], device="cuda"), pos=torch.arange(T, device="cuda") + 100,
                 freq=(100.0 ** (-torch.arange(0, D, 2, device="cuda").double() / D)).float(), heads=heads, D=D,
                 cu=torch.tensor([0, 70, T], dtype=torch.int32, device="cuda"))
    return leaves, fixed


def _run(f, leaves, fixed, gy, gs):
    y, s = _layer(f, leaves["H"], leaves["w"], leaves, fixed["decay"], fixed["pos"], fixed["freq"], fixed["heads"], fixed["D"],
                  fixed["cu"], leaves["s0"])
    return y, s, torch.autograd.grad([y, s], list(leaves.values()), [gy.to(y.dtype), gs.to(s.dtype)])


@pytest.mark.parametrize("dt,bar", [(torch.float32, 2e-5), (torch.bfloat16, 4e-2)])
def test_training_graph_gradients(A, dt, bar):
    """Every leaf's gradient through the whole layer against float64 autograd
    of the plain operations, in the 2-norm: fp32 within 2e-5 (some 200
    operations deep at 2^-23); bf16 within ten roundings of 2^-8 on each of
    the paths a gradient takes (qkv, q and k, o, their gradients, dz)."""
    from depth_wise_attention_block_gb300 import autograd as F
    leaves, fixed = _leaves(dt, 4)
    g = torch.Generator(device="cuda").manual_seed(9)
    gy, gs = torch.randn(200, 128, generator=g, device="cuda").to(dt), torch.randn(2, 2, 64, 64, generator=g, device="cuda")
    y, s, grads = _run(F, leaves, fixed, gy, gs)
    ref = {k: v.detach().double().requires_grad_() for k, v in leaves.items()}
    ry, rs, rgrads = _run(_Plain, ref, fixed, gy.double(), gs.double())
    for name, got, want in [("y", y, ry), ("s", s, rs)] + [(n, a, b) for n, a, b in zip(leaves, grads, rgrads)]:
        rel = float((got.detach().double() - want.detach()).norm() / want.detach().norm())
        assert torch.isfinite(got).all() and rel <= bar, (name, rel)


def test_training_graph_gradients_are_the_differences(A):
    """fp32 gradients against central differences of the float64 loss along
    random directions (whose rounding is 1e-16 / 1e-6 of the loss)."""
    from depth_wise_attention_block_gb300 import autograd as F
    leaves, fixed = _leaves(torch.float32, 5)
    g = torch.Generator(device="cuda").manual_seed(2)
    gy, gs = torch.randn(200, 128, generator=g, device="cuda"), torch.randn(2, 2, 64, 64, generator=g, device="cuda")
    _, _, grads = _run(F, leaves, fixed, gy, gs)

    def loss(ls):
        y, s = _layer(_Plain, ls["H"], ls["w"], ls, fixed["decay"], fixed["pos"], fixed["freq"], fixed["heads"], fixed["D"],
                      fixed["cu"], ls["s0"])
        return float((y * gy).sum() + (s * gs).sum())
    base = {k: v.detach().double() for k, v in leaves.items()}
    for (name, v), grad in zip(base.items(), grads):
        u = torch.randn(v.shape, generator=g, device="cuda").double()
        h = 1e-6
        up, dn = loss({**base, name: v + h * u}), loss({**base, name: v - h * u})
        want = (up - dn) / (2 * h)
        got = float((grad.double() * u).sum())
        scale = float(grad.double().norm() * u.norm())
        assert abs(got - want) <= 2e-5 * scale, (name, got, want)


def test_a_backward_can_be_captured(A):
    """Gradients written by a captured forward and backward, replayed on new
    inputs, are the eager ones."""
    from depth_wise_attention_block_gb300 import autograd as F
    leaves, fixed = _leaves(torch.bfloat16, 6)
    gy, gs = torch.randn(200, 128, device="cuda").bfloat16(), torch.randn(2, 2, 64, 64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(F, leaves, fixed, gy, gs)  # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, _, grads = _run(F, leaves, fixed, gy, gs)
    gy.normal_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in grads]
    _, _, want = _run(F, leaves, fixed, gy, gs)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_gradients_nobody_asks_for(A):
    from depth_wise_attention_block_gb300 import autograd as F
    x = torch.randn(2, 5, 24, device="cuda", requires_grad=True)
    w = torch.randn(7, 24, device="cuda")
    y = F.linear(x, w, residual=torch.randn(2, 5, 7, device="cuda"), activation="gelu")
    assert y.shape == (2, 5, 7)
    y.sum().backward()
    assert x.grad.shape == x.shape and w.grad is None
    q = torch.randn(6, 2, 16, device="cuda", requires_grad=True)
    v = torch.randn(6, 2, 16, device="cuda")
    out, _ = F.linear_attention(q, v, v, torch.zeros(2, device="cuda"))
    out.sum().backward()
    assert torch.isfinite(q.grad).all()
    with pytest.raises(ValueError, match="constant"):
        F.linear_attention(q, v, v, torch.zeros(2, device="cuda", requires_grad=True))
