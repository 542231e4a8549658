"""A workspace kept for the largest batch serves every smaller one."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def test_sizes_grow_with_tokens_and_sequences(A):
    rng = random.Random(1)
    for size in (A.attnres_linear_attention_workspace_size, A.attnres_linear_attention_backward_workspace_size):
        for _ in range(3000):
            T, n, H = int(2 ** rng.uniform(0, 18)), int(2 ** rng.uniform(0, 10)), rng.choice([1, 2, 8, 24, 32, 56, 64])
            Dk, Dv = rng.choice([(128, 128), (64, 64), (64, 128), (40, 24), (96, 96), (256, 256), (1, 1)])
            dt = rng.choice([torch.bfloat16, torch.float32])
            less = size(rng.randint(0, T), H, Dk, Dv, dt, rng.randint(1, n))
            assert 0 <= less <= size(T, H, Dk, Dv, dt, n)


@pytest.mark.parametrize("dt,D,H,T", [(torch.bfloat16, 64, 32, 16384), (torch.float32, 40, 64, 4096)])
def test_one_buffer_for_all_batches(A, dt, D, H, T):
    """Many sequences fill the GPU by themselves and are not cut; fewer, or
    shorter ones, are: the buffer of the first serves the others, with the same
    bits as one of their own."""
    most = 256
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn((T, H, D), generator=g, device="cuda").to(dt) for _ in range(4))
    decay = -torch.rand(H, generator=g, device="cuda")
    size = max(A.attnres_linear_attention_workspace_size(T, H, D, D, dt, most),
               A.attnres_linear_attention_backward_workspace_size(T, H, D, D, dt, most))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for n, t in [(most, T), (T // 256, T), (T // 400, T), (5, T), (1, T), (1, T // 9), (most, T // 7), (most, most), (1, 1)]:
        cu = torch.linspace(0, t, n + 1, device="cuda").int()
        results = []
        for w in (ws, None):
            out, fin = torch.empty_like(v[:t]), torch.empty(n, H, D, D, device="cuda")
            grads = [torch.empty_like(v[:t]) for _ in range(3)]
            A.attnres_linear_attention(q[:t], k[:t], v[:t], decay, out, cu_seqlens=cu, final_state=fin, workspace=w)
            A.attnres_linear_attention_backward(q[:t], k[:t], v[:t], decay, do[:t], *grads, cu_seqlens=cu, workspace=w)
            results.append([out, fin, *grads])
        assert all(torch.equal(a, b) for a, b in zip(*results)), (n, t)
