"""The gated recurrence over batches with padding ahead of the first sequence
and behind the last, cut inside tiles: whatever the padding holds (NaN and
infinities too), the sequences' results have the same bits, and nothing is
written to the padding's rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def _call(A, x, f, g, dy, cu, s0, ds1, T, C, dt):
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out, dx, df, dg = torch.full((4, T, C), 7.0, dtype=dt, device="cuda")
    fin, ds0 = torch.zeros_like(s0), torch.zeros_like(s0)
    chunk = torch.full((-(-T // 64), C), float("nan"), device="cuda")
    A.attnres_gated_recurrence(x, f, out, gate=g, cu_seqlens=cut, initial_state=s0, final_state=fin, chunk_states=chunk)
    A.attnres_gated_recurrence_backward(x, f, chunk, dy, dx, df, dg if g is not None else None, gate=g, cu_seqlens=cut, initial_state=s0,
                                        grad_final_state=ds1, grad_initial_state=ds0)
    return [out, dx, df] + ([dg] if g is not None else []), [fin, ds0]


# cuts inside the first and the last tile, inside one warp's rows, one row in
# from either end, between whole tiles of padding, all rows in one tile
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("T,C,cu", [(2000, 512, [37, 700, 700, 1950]), (64, 64, [3, 40]), (700, 72, [1, 699]), (1500, 1000, [130, 131, 1203, 1210]),
                                    (3000, 2048, [5, 1000, 2991]), (640, 136, [320, 321]), (200, 7, [9, 190])])
def test_padding_is_neither_read_into_results_nor_written(A, T, C, cu, gate, dt):
    gen = torch.Generator(device="cuda").manual_seed(T + C)
    n = len(cu) - 1
    x, f, g, dy = torch.randn(4, T, C, generator=gen, device="cuda").to(dt)
    s0, ds1 = torch.randn(2, n, C, generator=gen, device="cuda")
    g = g if gate else None
    live = torch.zeros(T, dtype=torch.bool, device="cuda")
    live[cu[0]:cu[-1]] = True
    rows, states = _call(A, x, f, g, dy, cu, s0, ds1, T, C, dt)
    for t in rows:
        assert torch.isfinite(t[live]).all() and (t[~live] == 7).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        ins = [None if t is None else t.clone() for t in (x, f, g, dy)]
        for t in ins:
            if t is not None:
                t[~live] = bad
        for _ in range(3):
            rows2, states2 = _call(A, *ins, cu, s0, ds1, T, C, dt)
            for a, b in zip(rows2 + states2, rows + states):
                assert torch.equal(a, b)
