"""A layer body between forwards, as a serving loop uses it: rows that become
padding, and a capture that leaves the states as they were."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _make(T, n, decode, dt, D=64, heads=2, d=128, L=3, seed=1, index=None):
    """(body, stack, states) with `index` as the slots or the offsets."""
    from depth_wise_attention_block_gb300.bodies import LinearAttentionBody, LinearAttentionWeights
    from depth_wise_attention_block_gb300.stack import StackForward
    g = torch.Generator(device="cuda").manual_seed(seed)
    layers = [LinearAttentionWeights(w_qkv=_normal(g, heads * 3 * D, d, scale=d ** -0.5, dtype=dt),
                                     w_out=_normal(g, d, heads * D, scale=(heads * D) ** -0.5, dtype=dt),
                                     b_out=_normal(g, d, scale=0.1)) for _ in range(L)]
    states = _normal(g, L, n, heads, D, D)
    decay = -torch.tensor([0.5, 0.01], device="cuda")
    kw = dict(decode=True, slots=index) if decode else dict(cu_seqlens=index)
    body = LinearAttentionBody(layers, T, heads, D, D, decay, states, **kw)
    h0, W = _normal(g, T, d, dtype=dt), _normal(g, L + 1, d, scale=1 / math.sqrt(d))
    return body, StackForward(h0, W, None, None, L, 2, body=body, keep_weights=False), states


def _index(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("decode,T,n,first,then,dead", [
    (True, 5, 4, (2, 0, -1, 3, 1), (2, -1, 0, 3, 4), [1, 4]),
    (False, 300, 2, (0, 120, 300), (10, 100, 250), [*range(10), *range(250, 300)]),
    (False, 40, 3, (0, 10, 20, 40), (0, 0, 0, 0), [*range(40)]),
])
def test_rows_that_become_padding_give_the_bias(A, decode, T, n, first, then, dead, dt, captured):
    """v = b_out wherever no sequence is: an exact zero times W_out, plus the
    bias, rounded.  The other rows are those of a body that never knew the
    first offsets."""
    index = _index(*first)
    body, fwd, states = _make(T, n, decode, dt, index=index)
    start = states.clone()
    if captured:
        fwd.capture()
    fwd.run()
    index.copy_(_index(*then))
    states.copy_(start)
    r = fwd.run().clone()
    want = body.layers[-1].b_out.to(dt)
    assert (fwd.F[dead] == want).all()
    _, fresh, fresh_states = _make(T, n, decode, dt, index=_index(*then))
    assert torch.equal(fresh.run(), r) and torch.equal(fresh.F, fwd.F) and torch.equal(fresh_states, states)


def test_rows_that_become_padding_on_another_stream(A):
    index, side = _index(1, 0, 2), torch.cuda.Stream()
    body, fwd, states = _make(3, 3, True, torch.bfloat16, index=index)
    for stream in (side, side.cuda_stream):
        index.copy_(_index(1, 0, 2))
        torch.cuda.synchronize()
        fwd.run(stream=stream)
        torch.cuda.synchronize()
        index.copy_(_index(1, -1, 2))
        torch.cuda.synchronize()
        fwd.run(stream=stream)
        torch.cuda.synchronize()
        assert (fwd.F[1] == body.layers[-1].b_out.bfloat16()).all()


def test_rows_that_become_padding_in_a_chunk_of_layers(A):
    """A pipeline stage issues some of the layers only."""
    index = _index(1, 0, 2)
    body, fwd, _ = _make(3, 3, True, torch.bfloat16, index=index)
    r, F = torch.randn(3, 128, device="cuda").bfloat16(), torch.empty(3, 128, device="cuda", dtype=torch.bfloat16)
    for layer in (2, 3):
        body.issue(layer, r, F)
    index.copy_(_index(1, -1, 2))
    for layer in (2, 3):
        body.issue(layer, r, F)
        assert (F[1] == body.layers[layer - 1].b_out.bfloat16()).all()


@pytest.mark.parametrize("schedule", ["single", "hybrid"])
@pytest.mark.parametrize("decode,T,n,index,dt,D", [
    (True, 5, 5, None, torch.bfloat16, 64), (True, 5, 8, (7, 1, -1, 3, 1), torch.bfloat16, 128), (True, 3, 3, None, torch.float32, 24),
    (False, 70, 1, None, torch.bfloat16, 64), (False, 300, 3, (0, 0, 120, 300), torch.bfloat16, 128),
    (False, 6000, 1, None, torch.bfloat16, 128), (False, 6000, 2, (0, 90, 6000), torch.bfloat16, 64),
    (False, 6000, 2, (0, 90, 6000), torch.float32, 24), (False, 200, 1, None, torch.float32, 24),
])
def test_capture_leaves_the_states(A, decode, T, n, index, dt, D, schedule):
    """Recording a forward is not running one: the states after capture() are
    the bits before it (an infinity and a NaN among them), and the first
    replay is the first forward."""
    index = None if index is None else _index(*index)
    body, fwd, states = _make(T, n, decode, dt, D=D, index=index)
    fwd_kw = dict(schedule=schedule, two_phase_from=2, keep_weights=False)
    from depth_wise_attention_block_gb300.stack import StackForward
    fwd = StackForward(fwd.state.h0, fwd.W, None, None, 3, 2, body=body, **fwd_kw)
    start = states.clone()
    odd = start.clone()
    odd.view(-1)[3], odd.view(-1)[7] = float("inf"), float("nan")
    states.copy_(odd)
    fwd.capture()
    torch.cuda.synchronize()
    assert torch.equal(states.view(torch.int32), odd.view(torch.int32))
    assert (body.slots if decode else body.cu_seqlens) is index
    states.copy_(start)
    got = [(fwd.run().clone(), states.clone()) for _ in range(2)]
    states.copy_(start)
    eager = StackForward(fwd.state.h0, fwd.W, None, None, 3, 2, body=body, **fwd_kw)
    for r, s in got:
        assert torch.equal(eager.run(), r) and torch.equal(states, s)
