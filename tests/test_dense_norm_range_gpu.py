"""The norm at the ends of fp32's range against the formula in fp64: an eps beside squares
that are finite by themselves, and small values in rows whose squares are not."""
import numpy as np
import pytest
import torch

import dense_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
MOST = float(np.finfo(np.float32).max)


def _tol(want, half_step=0.0):
    """As for the norm at ordinary sizes: 28 roundings of 2^-24 each, 32 counted, and the output's own; the least fp32 value
    where an intermediate is subnormal."""
    return (32 * 2.0 ** -24 + half_step) * np.abs(want) + 2.0 ** -148


@pytest.mark.parametrize("C,top", [(1, 1.5e19), (2, 1.2e19), (3, 1e19), (7, 6.5e18), (8, 6.4e18), (100, 1e18), (128, 1e18), (130, 1e18),
                                   (512, 5e17), (520, 5e17), (4096, 2e17), (12290, 1e17), (32768, 5e16)])
def test_eps_beside_finite_squares(C, top):
    """The sum of squares is finite, and so is eps, but not the mean and eps together."""
    x = torch.full((5, C), top)
    x[:, ::2] *= -1
    x[1] *= 0.5
    x[2] *= 1e-3
    w = torch.linspace(0.5, 2.0, C)
    for eps in (3e38, MOST):
        eps = float(np.float32(eps))
        _, want = ref.norm(x.double().numpy(), None, w.double().numpy(), eps)
        y, _ = kda.kda_add_rmsnorm(x.cuda(), None, w.cuda(), eps)
        assert (np.abs(y.double().cpu().numpy() - want) <= _tol(want)).all()
        s, want = ref.norm(x.double().numpy(), x.double().numpy() * 0.25, w.double().numpy(), eps)
        y, h = kda.kda_add_rmsnorm(x.cuda(), 0.25 * x.cuda(), w.cuda(), eps)
        assert (np.abs(y.double().cpu().numpy() - want) <= _tol(want)).all()
        codes, scales, _ = kda.kda_add_rmsnorm_fp8(x.cuda(), None, w.cuda(), eps)
        v = kda.kda_fp8_values(codes, scales, 1, torch.float32).double().cpu().numpy()
        _, want = ref.norm(x.double().numpy(), None, w.double().numpy(), eps)
        # E4M3: half a step of 2^-4, or of the least step under the block's scale (2^-10 of it, 448 of which hold the largest)
        assert (np.abs(v - want) <= (2.0 ** -4 + 2.0 ** -19) * np.abs(want) + 2.0 ** -10 * np.abs(want).max(1, keepdims=True) / 224).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C", [4, 27, 64, 128, 130, 300, 520, 4096, 12290])
def test_small_values_beside_squares_beyond_the_range(C, dt):
    """Rows whose squares overflow through one value: the others, up to 2^128 below it, keep their precision (bf16's subnormal
    results are off by 2^-134 at most)."""
    g = torch.Generator().manual_seed(C)
    x = torch.randn(6, C, generator=g, dtype=torch.float64)
    for i, e in enumerate((0, -20, -50, -60, -62, -63)):
        x[i] *= 2.0 ** e
    x[:, C // 2] = 2.0 ** 64 * C ** 0.5
    x = x.to(dt)
    _, want = ref.norm(x.double().numpy(), None, None, 1e-6)
    y, _ = kda.kda_add_rmsnorm(x.cuda())
    half, least = (2.0 ** -8, 2.0 ** -134) if dt is torch.bfloat16 else (0.0, 0.0)
    assert (np.abs(y.double().cpu().numpy() - want) <= _tol(want, half) + least).all()
