"""Every cut of the 8-bit product on the GPU, given by name, against exact sums."""
import pytest
import torch

import dense_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda
from test_dense_matmul_gpu import _dense, _exact_operands

pytestmark = pytest.mark.gpu

CUTS = [(rows, split, deep) for rows in (16, 32, 64, 128, 256) for split in (1, 2, 4, 8) for deep in ((0, 1) if rows < 256 else (1,))] + [(0, 1, 1)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cut", CUTS)
def test_every_cut(cut, dt, monkeypatch):
    """One token, tokens that end inside a tile and past one, K of uneven parts, and columns that end inside four."""
    t = torch.float32 if dt == "f32" else torch.bfloat16
    ref.force_cut(monkeypatch, lambda *_: cut)
    rows = cut[0] or 256
    for M, N, K in ((1, 300, 4096), (rows - 1, 129, 4640), (2 * rows + 3, 514, 5136), (rows + 1, 1023, 7696)):
        if cut[1] > -(-K // 512):
            continue
        a, sa, w, sw = (x.cuda() for x in _exact_operands(M, N, K, M + N))
        want = (_dense(a, sa, 1) @ _dense(w, sw, 128).t()).to(t)
        assert torch.equal(kda.kda_fp8_matmul(a, sa, w, sw, t), want), (M, N, K)
        big = torch.full((M, N + 3), -5.0, device="cuda", dtype=t)
        kda.kda_fp8_matmul(a, sa, w, sw, out=big[:, 1:1 + N])
        assert torch.equal(big[:, 1:1 + N], want) and (big[:, :1] == -5).all() and (big[:, 1 + N:] == -5).all(), (M, N, K)
    assert kda.kda_device_error() == (0, 0)


def test_the_environment_does_not_choose(monkeypatch):
    """More rows than a grid has tiles of 256 (an inherited KDA_FP8_PAIR=0 once made such calls fail)."""
    monkeypatch.setenv("KDA_FP8_PAIR", "0")
    M = 65535 * 256 + 1
    a = torch.zeros(M, 16, device="cuda", dtype=torch.uint8)
    a[:, 0] = torch.arange(M, device="cuda").remainder(7) * 8      # codes of 0, 2^-6, 2^-5, ...
    a = a.view(torch.float8_e4m3fn)
    one = torch.full((1, 16), 1.0, device="cuda").to(torch.float8_e4m3fn)
    got = kda.kda_fp8_matmul(a, torch.full((M, 1), 127, dtype=torch.uint8, device="cuda"), one, torch.full((1, 1), 127, dtype=torch.uint8, device="cuda"))
    assert torch.equal(got[:, 0], a[:, 0].to(torch.bfloat16))


def _operands(M, N, K):
    """Rows and columns over some powers of two, so that the order of a sum shows in its bits."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M, K, device="cuda", generator=g) * torch.exp(2 * torch.randn(M, K, device="cuda", generator=g))
    return (*kda.kda_fp8_quant(x), *kda.kda_fp8_quant(torch.randn(N, K, device="cuda", generator=g), 128))


@pytest.mark.parametrize("M,N,K", [(39, 6169, 7184), (55, 4345, 6448), (61, 4955, 9888), (1, 16416, 4096), (228, 16300, 4096), (974, 4516, 912),
                                   (64, 4096, 12288)])
def test_bf16_is_fp32_rounded(M, N, K):
    """Sizes at which the two types would be cut differently among them."""
    ops = _operands(M, N, K)
    f, h = kda.kda_fp8_matmul(*ops, torch.float32), kda.kda_fp8_matmul(*ops)
    assert torch.equal(f.bfloat16(), h)


@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_bits_depend_on_the_parts_of_k_alone(split, monkeypatch):
    ops = _operands(130, 513, 4112)
    got = []
    for cut in CUTS:
        if cut[1] == split:
            with monkeypatch.context() as m:
                ref.force_cut(m, lambda *_: cut)
                got.append(kda.kda_fp8_matmul(*ops, torch.float32))
    assert len(got) >= 9 and all(torch.equal(got[0], f) for f in got)
