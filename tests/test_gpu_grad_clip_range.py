"""attnres_grad_clip where max_norm / norm, or the norm itself, leaves fp32,
against its fp64 statement.

Tolerances, derived before any run: the norm is off by 19 2^-24 of itself and a
value by that, three fp32 roundings, its own (u: bf16 2^-8, fp32 2^-24) and a
step of the type's smallest number (bf16 2^-133, fp32 2^-149)."""
import numpy as np
import pytest
import torch

from oracle import body_oracle as B

pytestmark = pytest.mark.gpu
N_ERR = 19 * 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
STEP = {torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}
FLT_MAX = float(np.finfo(np.float32).max)
# single elements ahead of a boundary, whole vectors, several chunks, tails
SIZES = [1, 7, 4096, 70001, 9]


@pytest.fixture(scope="module")
def A():
    import depth_wise_attention_block_gb300 as A
    return A


def to64(t):
    return t.detach().double().cpu().numpy()


def _grads(dts, scale, shift=0):
    g = torch.Generator(device="cuda").manual_seed(shift)
    return [(torch.randn(n + shift, generator=g, device="cuda").clamp_(-3, 3) * scale).to(dts[i % len(dts)])[shift:]
            for i, n in enumerate(SIZES)]


def _check(A, grads, max_norm, outs=None):
    max_norm = float(np.float32(max_norm))
    want_norm, want = B.grad_clip([to64(t) for t in grads], max_norm)
    norm = torch.zeros(1, device="cuda")
    A.attnres_grad_clip(grads, max_norm, norm, outs=outs)
    for t, w in zip(grads if outs is None else outs, want):
        bound = (U[t.dtype] + N_ERR + 3 * 2.0 ** -24) * np.abs(w) + STEP[t.dtype]
        err = np.abs(to64(t) - w)
        assert (err <= bound).all(), f"worst {(err / bound).max():.3g} x bound"
    return float(norm), want_norm


DTYPES = [(torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)]


@pytest.mark.parametrize("dts", DTYPES)
@pytest.mark.parametrize("max_norm", [1e-2, 1e-6, 1e-9, 1e-20, 1e-35, 1e-40])
def test_a_ratio_below_fp32(A, dts, max_norm):
    """Gradients of 1e35: max_norm / norm of 1e-40 to 1e-78, results that are
    ordinary numbers (and, for the last bounds, near the types' smallest)."""
    for shift in (0, 1):
        grads = _grads(dts, 1e35, shift)
        for outs in ([torch.full_like(t, 5.0) for t in grads], None):
            norm, want = _check(A, grads, max_norm, outs)
            assert abs(norm - want) <= N_ERR * want


@pytest.mark.parametrize("dts", DTYPES)
@pytest.mark.parametrize("scale", [1e-37, 1e-34])
def test_small_gradients_keep_their_digits(A, dts, scale):
    """Results near fp32's smallest normal number, and below it."""
    for max_norm in (1e-1 * scale, 1e-3 * scale, 1e-6 * scale):
        grads = _grads(dts, scale)
        norm, want = _check(A, grads, max_norm, [torch.empty_like(t) for t in grads])
        assert abs(norm - want) <= N_ERR * want + 2.0 ** -149


@pytest.mark.parametrize("dts", DTYPES)
@pytest.mark.parametrize("max_norm", [1e38, 1.0, 1e-6])
def test_a_norm_above_fp32(A, dts, max_norm):
    """Finite gradients whose norm fp32 does not hold are clipped; the norm is
    reported as fp32's largest number, so infinity and NaN still say that
    nothing was scaled."""
    grads = _grads(dts, 1e38)
    norm, want = _check(A, grads, max_norm, [torch.empty_like(t) for t in grads])
    assert want > 1e40 and norm == FLT_MAX
    alone = torch.zeros(1, device="cuda")
    before = [t.clone() for t in grads]
    A.attnres_grad_clip(grads, float("inf"), alone)
    assert float(alone) == FLT_MAX and all(torch.equal(t, b) for t, b in zip(grads, before))
    grads[2][5] = float("inf")
    before = [t.clone() for t in grads]
    A.attnres_grad_clip(grads, max_norm, alone)
    assert float(alone) == float("inf") and all(torch.equal(t, b) for t, b in zip(grads, before))
