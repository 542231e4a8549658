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
