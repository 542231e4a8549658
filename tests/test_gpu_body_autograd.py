"""The differentiable operators of a layer body as a training program may use
them: buffers written again, gradients of some inputs only."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    from depth_wise_attention_block_gb300 import autograd as F
    return F


def _randn(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def _rope(F, T=12, D=64):
    q, k = _randn(1, T, 4, D).requires_grad_(), _randn(2, T, 2, D).requires_grad_()
    pos = torch.arange(T, device="cuda")
    freq = 100.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    return q, k, pos, freq


@pytest.mark.parametrize("which", ["positions", "inv_freq"])
def test_angles_written_before_the_backward(F, which):
    """The backward needs the forward's angles: torch says so when they are gone."""
    q, k, pos, freq = _rope(F)
    a, b = F.qk_norm_rope(q, k, positions=pos, inv_freq=freq)
    (pos if which == "positions" else freq).add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        (a.sum() + b.sum()).backward()


def test_angles_kept_give_the_gradients(F):
    """The same bits as the call's own backward."""
    import depth_wise_attention_block_gb300 as A
    q, k, pos, freq = _rope(F)
    ga, gb = _randn(3, *q.shape), _randn(4, *k.shape)
    got = torch.autograd.grad(F.qk_norm_rope(q, k, positions=pos, inv_freq=freq), (q, k), (ga, gb))
    want = [torch.empty_like(q), torch.empty_like(k)]
    with torch.no_grad():
        A.attnres_qk_norm_rope_backward(q, k, ga, gb, *want, positions=pos, inv_freq=freq)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_frequencies_get_no_gradient(F):
    """Refused, not left out."""
    q, k, pos, freq = _rope(F)
    with pytest.raises(ValueError, match="constant"):
        F.qk_norm_rope(q, k, positions=pos, inv_freq=freq.requires_grad_())


E = 2.0 ** -23


@pytest.mark.parametrize("dt,T,D", [(torch.float32, 150, 24), (torch.bfloat16, 200, 64), (torch.bfloat16, 6000, 64), (torch.float32, 6000, 24)])
@pytest.mark.parametrize("need", [c for n in (1, 2, 3) for c in itertools.combinations("qkvs", n)])
def test_attention_gradients_of_some_inputs(F, monkeypatch, dt, T, D, need):
    """Those asked for are the formula's; the others are not formed (grad_v
    is, where the initial state's gradient comes out of its scan)."""
    import numpy as np
    from oracle import body_oracle as B
    H, n = 2, 2
    x = dict(q=_randn(1, T, H, D, dtype=dt), k=_randn(2, T, H, D, dtype=dt), v=_randn(3, T, H, D, dtype=dt), s=_randn(4, n, H, D, D))
    for name in need:
        x[name].requires_grad_()
    cu = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    g = -torch.tensor([0.02, 0.4], device="cuda")
    do, ds = _randn(5, T, H, D, dtype=dt), _randn(6, n, H, D, D)
    asked = []
    call = F.attnres_linear_attention_backward

    def spy(q, k, v, log_decay, grad_out, grad_q, grad_k, grad_v, **kw):
        asked.append("".join(name for name, t in zip("qkvs", (grad_q, grad_k, grad_v, kw["grad_initial_state"])) if t is not None))
        return call(q, k, v, log_decay, grad_out, grad_q, grad_k, grad_v, **kw)
    monkeypatch.setattr(F, "attnres_linear_attention_backward", spy)
    got = torch.autograd.grad(F.linear_attention(x["q"], x["k"], x["v"], g, cu, x["s"]), [x[name] for name in need], [do, ds])
    assert asked == ["".join(name for name in "qkvs" if name in need or (name == "v" and "s" in need))]

    def to64(t):
        return t.detach().double().cpu().numpy()
    args = [to64(x[name]) for name in "qkv"]
    cu64 = to64(cu).astype(int)
    want = B.linear_attention_backward(*args, to64(g), cu64, to64(x["s"]), D ** -0.5, to64(do), to64(ds))
    cond = B.linear_attention_backward(*[np.abs(a) for a in args], to64(g), cu64, np.abs(to64(x["s"])), D ** -0.5,
                                       np.abs(to64(do)), np.abs(to64(ds)))
    # sums over channels and tokens in fp32, the scores and the state rounded to bf16, the result rounded
    u = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
    for name, t in zip(need, got):
        i = "qkvs".index(name)
        bound = (T + 64) * E * cond[3] if name == "s" else \
            u * np.abs(want[i]) + ((2 * D + T + 64) * E + (2 * u if dt == torch.bfloat16 else 0)) * cond[i]
        err = np.abs(to64(t) - want[i])
        assert np.isfinite(err).all() and (err <= bound + 2.0 ** -129).all(), (name, (err / bound).max())


def test_attention_backward_of_nothing_and_its_refusals():
    """Without an output there is nothing to do; the initial state's gradient
    needs grad_v's scan."""
    import depth_wise_attention_block_gb300 as A
    q = _randn(1, 10, 2, 16)
    s, g = torch.zeros(1, 2, 16, 16, device="cuda"), torch.zeros(2, device="cuda")
    A.attnres_linear_attention_backward(q, q, q, g, q, None, None, None)
    with pytest.raises(A.AttnresError, match="grad_v"):
        A.attnres_linear_attention_backward(q, q, q, g, q, torch.empty_like(q), torch.empty_like(q), None, grad_initial_state=s)


@pytest.mark.parametrize("need", [c for n in (1, 2, 3) for c in itertools.combinations(range(4), n)])
@pytest.mark.parametrize("D", [64, 37])
def test_rope_gradients_of_some_inputs(F, monkeypatch, D, need):
    """The same bits as with all of them (a gain's, whose partial sums depend
    on the launch, within 128 fp32 operations of its sum); a tensor whose
    gradient, and whose gain's, nobody asks for does not go through the call."""
    def leaves():
        return [_randn(1, 12, 4, D), _randn(2, 12, 2, D), _randn(3, D), _randn(4, D)]

    def grads(which):
        x = leaves()
        for i in which:
            x[i].requires_grad_()
        outs = F.qk_norm_rope(*x)
        on = [o for o in outs if o.requires_grad]
        return torch.autograd.grad(outs, [x[i] for i in which], [_randn(5, 12, 4, D), _randn(6, 12, 2, D)]) if len(on) == 2 else None
    full = grads(range(4))
    asked = []
    call = F.attnres_qk_norm_rope_backward

    def spy(q, k, *a, **kw):
        asked.append((q is not None, k is not None))
        return call(q, k, *a, **kw)
    monkeypatch.setattr(F, "attnres_qk_norm_rope_backward", spy)
    got = grads(need)
    assert asked == [(bool({0, 2} & set(need)), bool({1, 3} & set(need)))]
    x = leaves()
    for i, t in zip(need, got):
        if i < 2:
            assert torch.equal(t, full[i])
        else:
            hat = x[i - 2] * torch.rsqrt(x[i - 2].square().mean(-1, keepdim=True) + 1e-5)
            cond = (_randn(3 + i, 12, x[i - 2].shape[1], D) * hat).abs().sum((0, 1))
            assert ((t - full[i]).abs() <= 128 * E * cond).all()


@pytest.mark.parametrize("dt,T,D", [(torch.float32, 150, 24), (torch.bfloat16, 200, 64), (torch.bfloat16, 6000, 64), (torch.float32, 6000, 24),
                                    (torch.bfloat16, 6000, 128), (torch.float32, 0, 24), (torch.bfloat16, 0, 64)])
def test_state_gradient_in_place_without_the_others(dt, T, D):
    """grad_initial_state over grad_final_state, with grad_v only: the same bits
    as apart (no rows: with no other output at all), empty sequences among
    them."""
    import depth_wise_attention_block_gb300 as A
    H, n = 2, 4
    q, k, v, do = (_randn(i, T, H, D, dtype=dt) for i in range(4))
    cu = torch.tensor([0, T // 3, T // 3, T, T], dtype=torch.int32, device="cuda")
    g, ds = -torch.tensor([0.02, 0.4], device="cuda"), _randn(5, n, H, D, D)
    apart, over = torch.empty_like(ds), ds.clone()
    gv = [torch.empty_like(v) if T else None for _ in range(2)]
    A.attnres_linear_attention_backward(q, k, v, g, do, None, None, gv[0], cu_seqlens=cu, grad_final_state=ds, grad_initial_state=apart)
    A.attnres_linear_attention_backward(q, k, v, g, do, None, None, gv[1], cu_seqlens=cu, grad_final_state=over, grad_initial_state=over)
    assert torch.equal(apart, over) and torch.isfinite(over).all()
    assert torch.equal(over[[1, 3]], ds[[1, 3]])
    if T:
        assert torch.equal(gv[0], gv[1])
    else:
        assert torch.equal(over, ds)
