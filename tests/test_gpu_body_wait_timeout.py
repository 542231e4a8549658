"""The timeout path of the bounded waits in the layer body's kernels, exercised
on a healthy GPU (as in test_gpu_wait_timeout.py): attnres_debug_wait_test makes
every CTA arm its first block or tile without issuing its copies and limits the
main-loop waits.  The call must set ATTNRES_DEVERR_WAIT_TIMEOUT, write NaN,
drain what it did issue and return; after (0, -1) the same call gives the same
bits as before.  Nothing here faults or hangs a GPU: every wait is bounded and
every issued copy targets valid memory and is waited for before the CTA exits.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

LIMIT_NS = 1_000_000   # 1 ms: far above any healthy copy's latency


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def _randn(seed, *shape, dtype):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def _check(A, call, outs):
    """`call(dev_err)` fills `outs`: right, withheld, right again."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    A.attnres_debug_wait_test(LIMIT_NS, 0)
    try:
        call(err)
        torch.cuda.synchronize()
    finally:
        A.attnres_debug_wait_test(0, -1)
    assert int(err.item()) & A.ATTNRES_DEVERR_WAIT_TIMEOUT
    for t in outs:
        assert torch.isnan(t).all()
    err.zero_()
    call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


# few rows (clusters; fp32: weights split on the way in, or made in memory
# first), single tiles, several per CTA, pairs of CTAs
@pytest.mark.parametrize("m,n,k,dt", [
    (16, 512, 2048, torch.bfloat16), (300, 1024, 1024, torch.bfloat16), (64, 21504, 256, torch.bfloat16),
    (2048, 7168, 512, torch.bfloat16), (4096, 2048, 1000, torch.bfloat16), (16, 512, 2048, torch.float32),
    (100, 512, 1024, torch.float32), (300, 1024, 512, torch.float32), (2048, 2048, 256, torch.float32)])
def test_linear_times_out_and_recovers(A, m, n, k, dt):
    x, w, out = _randn(1, m, k, dtype=dt), _randn(2, n, k, dtype=dt), torch.empty((m, n), dtype=dt, device="cuda")
    _check(A, lambda err: A.attnres_linear(x, w, out, activation="silu", dev_err=err), [out])


def test_linear_backward_times_out_and_recovers(A):
    dt = torch.bfloat16
    x, w, g = _randn(1, 512, 1024, dtype=dt), _randn(2, 768, 1024, dtype=dt), _randn(3, 512, 768, dtype=dt)
    gx, gw, gb = torch.empty_like(x), torch.empty_like(w), torch.empty(768, device="cuda")
    _check(A, lambda err: A.attnres_linear_backward(x, w, g, gx, gw, gb, activation="gelu", dev_err=err), [gx, gw, gb])


@pytest.mark.parametrize("T,H,D", [(300, 3, 128), (5000, 2, 128), (5000, 8, 64)])  # in one piece; in several
def test_linear_attention_times_out_and_recovers(A, T, H, D):
    q, k, v, do = (_randn(s, T, H, D, dtype=torch.bfloat16) for s in range(4))
    decay, s0 = torch.full((H,), -0.02, device="cuda"), _randn(5, 2, H, D, D, dtype=torch.float32)
    cu = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    out, fin = torch.empty_like(q), torch.empty_like(s0)
    _check(A, lambda err: A.attnres_linear_attention(q, k, v, decay, out, cu_seqlens=cu, initial_state=s0, final_state=fin, dev_err=err),
           [out, fin])
    grads, ds0 = [torch.empty_like(q) for _ in range(3)], torch.empty_like(s0)
    _check(A, lambda err: A.attnres_linear_attention_backward(q, k, v, decay, do, *grads, cu_seqlens=cu, initial_state=s0,
                                                              grad_initial_state=ds0, dev_err=err), [*grads, ds0])
