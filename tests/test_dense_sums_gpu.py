"""How exact the 8-bit product's fp32 sums are on uneven values, against fp64."""
import pytest
import torch

import linear_attention_recurrence_chunk_gb300 as kda
from test_dense_matmul_gpu import _dense

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 4096, 12288), (30, 513, 12288), (64, 4096, 12288), (250, 1000, 4096), (700, 1025, 512), (2048, 2052, 16384)])
def test_rms_of_the_error(M, N, K):
    """Rows and channels of uneven size.  Products are exact; each of the K / 32 instructions adds 32 of them to a sum S of 24
    bits.  Cut toward 0, which no rounding exceeds, that is off by 2^-24 |S| in the mean, always to the same side, and |S| is
    at most the row's rms in the mean: K / 32 2^-24 of it together.  As much again is counted for products that are cut
    where they are added and for the joins of partial sums.  (An output held in bf16 would be off by 2^-10 of it; the bound is
    2^-14.4 for K = 12,288.)"""
    g = torch.Generator(device="cuda").manual_seed(K + M)
    x = torch.randn(M, K, device="cuda", generator=g) * torch.exp(2 * torch.randn(M, 1, device="cuda", generator=g))
    y = torch.randn(N, K, device="cuda", generator=g) * torch.exp(torch.randn(1, K, device="cuda", generator=g))
    (a, sa), (w, sw) = kda.kda_fp8_quant(x, 1), kda.kda_fp8_quant(y, 128)
    want = _dense(a, sa, 1) @ _dense(w, sw, 128).t()
    f, h = kda.kda_fp8_matmul(a, sa, w, sw, torch.float32), kda.kda_fp8_matmul(a, sa, w, sw)
    rms = want.square().mean(1).sqrt()
    off = (f.double() - want).square().mean(1).sqrt() / rms
    print(f"rms of the error over the rms of a row, K = {K}: {off.max().item():.3g}, bound {K * 2.0 ** -28:.3g}")
    assert (off <= K / 32 * 2.0 ** -23).all()
    # one rounding on top: at most 2^-8 of a value, and of what the sum is off by
    assert ((h.double() - want).abs() <= 2.0 ** -8 * want.abs() + (f.double() - want).abs() * (1 + 2.0 ** -8)).all()
