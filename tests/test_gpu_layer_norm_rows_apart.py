"""Rows of a layer norm do not see one another where many rows share a CTA's
shared memory: infinities and NaN of some rows of x and of the incoming
gradient leave every other row's result as it was, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def _rows(seed, T, d, dt, wide):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, d + wide, generator=g, device="cuda").to(dt)[:, wide:]


def _run(A, x, dy, w, b):
    T, d = x.shape
    out, gx = torch.empty(2, T, d, dtype=x.dtype, device="cuda")
    gg, gb = torch.empty(2, d, device="cuda")
    A.attnres_layer_norm(x, out, gain=w, bias=b)
    A.attnres_layer_norm_backward(x, dy, gx, gain=w, grad_gain=gg, grad_bias=gb)
    alone = torch.empty_like(gx)
    A.attnres_layer_norm_backward(x, dy, alone, gain=w)
    return out, gx, gg, gb, alone


# widths that leave lanes without channels (in one warp, in the last of several,
# whole warps) beside ones that fill every lane; one row to a CTA, several, and
# many in turn; rows on the 16-byte vectors and off them; rows too wide for an SM
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("wide", [0, 1])
@pytest.mark.parametrize("T,d", [(3000, 8), (5000, 40), (3001, 136), (2000, 256), (2500, 520), (1500, 1000), (2003, 1024), (1999, 1032),
                                 (700, 2056), (900, 4104), (700, 7168), (500, 7176), (100, 1000), (152, 40), (153, 4104), (640, 20000)])
def test_other_rows_keep_their_bits(A, T, d, dt, wide):
    x, dy = _rows(1, T, d, dt, wide), _rows(2, T, d, dt, wide)
    w, b = _rows(3, 1, d, torch.float32, 0)[0], _rows(4, 1, d, torch.float32, 0)[0]
    want = _run(A, x, dy, w, b)
    assert all(torch.isfinite(t).all() for t in want)
    for trial in range(3):  # rows spread otherwise over the CTAs' turns
        bad_x = torch.unique(torch.tensor([0, 1, 7, T // 3, T // 2, T - 1] + list(range(trial, T, 41 + 12 * trial)), device="cuda"))
        bad_dy = torch.arange(5 + trial, T, 67, device="cuda")
        x2, dy2 = _rows(1, T, d, dt, wide), _rows(2, T, d, dt, wide)
        for i, v in enumerate((INF, NAN, -INF)):
            x2[bad_x[i::4], (i * d) // 4] = v
            dy2[bad_dy[i::4], (i * d) // 4] = v
        x2[bad_x[3::4]] = NAN       # padding of nothing but NaN, and of infinities
        dy2[bad_dy[3::4]] = INF
        out, gx, gg, gb, alone = _run(A, x2, dy2, w, b)
        sick = torch.zeros(T, dtype=torch.bool, device="cuda")
        sick[bad_x] = True
        assert torch.equal(out[~sick], want[0][~sick]) and torch.isnan(out[sick]).all()
        sick[bad_dy] = True
        assert torch.equal(gx[~sick], want[1][~sick]) and torch.equal(alone[~sick], want[4][~sick])
        assert not torch.isfinite(gx[sick]).any() and torch.isnan(gg).all()
        # the bias's gradient does not look at x
        only_x = _run(A, x2, dy, w, b)
        assert torch.equal(only_x[3], want[3])
