"""The product of 8-bit matrices on the GPU: exact on sums that fp32 holds exactly, and
against fp64 with the bound of an fp32 sum."""
import numpy as np
import pytest
import torch

import dense_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda

pytestmark = pytest.mark.gpu


def _blocks(n):
    return -(-n // 128)


def _exact_operands(M, N, K, seed):
    """Codes of whole numbers up to 8 and scales of 2^-1 .. 2^1: every partial sum is a multiple of 2^-2 below
    64 * 4 * K <= 2^22 for K up to 16,384, exact in fp32."""
    g = torch.Generator().manual_seed(seed)

    def codes(r):
        return torch.randint(-8, 9, (r, K), generator=g).float().to(torch.float8_e4m3fn)

    def scales(r):
        return torch.randint(126, 129, (r, _blocks(K)), generator=g, dtype=torch.int64).to(torch.uint8)

    return codes(M), scales(M), codes(N), scales(_blocks(N))


def _dense(codes, scales, rows):
    """fp64 values on the GPU (whole matrices of the larger cases)."""
    v = codes.double()
    T, C = v.shape
    return v * torch.exp2(scales.double() - 127).repeat_interleave(rows, 0)[:T].repeat_interleave(128, 1)[:, :C]


SIZES = [(1, 1, 16), (1, 128, 128), (1, 2052, 512), (3, 300, 1040), (8, 513, 4096), (16, 256, 4112), (17, 130, 144), (33, 1000, 1088), (64, 384, 640),
         (65, 129, 528), (100, 2052, 512), (128, 4096, 2048), (129, 640, 12288), (256, 513, 4096), (257, 384, 1040), (300, 2048, 272),
         (511, 1000, 512), (512, 1024, 1024), (777, 513, 2064), (1000, 2052, 512), (1024, 4096, 1024), (1500, 129, 16), (2049, 1111, 1152),
         (4096, 4096, 528), (3000, 5000, 2048),
         # each way of cutting the product that the choice by sizes has: rows of a tile, parts of K, one or two CTAs an SM
         (2, 6188, 2624), (42, 21, 15280), (1122, 514, 64), (52, 561, 15056), (6687, 62, 2784), (159, 2068, 6912), (1363, 54, 8800),
         (611, 16, 16048), (2357, 2519, 80), (6705, 108, 8864), (2749, 18, 11040), (1075, 7427, 2960), (10542, 19, 2496), (322, 8610, 48), (2657, 713, 14704), (1586, 400, 15472),
         (131, 2192, 11472), (138, 17775, 10368), (3758, 579, 14768), (2243, 84, 4336), (66, 5494, 11264),
         (5, 48, 1792), (655, 17, 3424), (11480, 258, 2000), (13258, 529, 3600), (5351, 16, 13632), (1, 4748, 15584), (2353, 36, 10080), (4683, 22, 11280),
         (2, 19561, 16160), (13994, 501, 7872)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_exact_sums(M, N, K, dt):
    """Every block's scale and every element in its place: the same bits as the exact sum, rounded once."""
    a, sa, w, sw = (t.cuda() for t in _exact_operands(M, N, K, M + N + K))
    want = _dense(a, sa, 1) @ _dense(w, sw, 128).t()
    t = torch.float32 if dt == "f32" else torch.bfloat16
    got = kda.kda_fp8_matmul(a, sa, w, sw, t)
    assert torch.equal(got, want.to(t))
    assert torch.equal(got, kda.kda_fp8_matmul(a, sa, w, sw, t))
    assert kda.kda_device_error() == (0, 0)


@pytest.mark.parametrize("pair", ["0", "1"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (5, 239, 512), (127, 241, 1040), (129, 480, 2064), (256, 8, 4096), (255, 1200, 528), (513, 1001, 272),
                                   (2304, 2160, 144), (700, 30000, 128)])
def test_both_kernels(M, N, K, dt, pair, monkeypatch):
    """Pairs of CTAs on small and ragged sizes, and single ones on large, against the exact sums."""
    monkeypatch.setenv("KDA_FP8_PAIR", pair)
    a, sa, w, sw = (t.cuda() for t in _exact_operands(M, N, K, M + N + K))
    want = _dense(a, sa, 1) @ _dense(w, sw, 128).t()
    t = torch.float32 if dt == "f32" else torch.bfloat16
    assert torch.equal(kda.kda_fp8_matmul(a, sa, w, sw, t), want.to(t))
    big = torch.full((M, N + 5), -5.0, device="cuda", dtype=t)         # rows that begin anywhere
    kda.kda_fp8_matmul(a, sa, w, sw, out=big[:, 2:2 + N])
    assert torch.equal(big[:, 2:2 + N], want.to(t)) and (big[:, :2] == -5).all() and (big[:, N + 2:] == -5).all()
    assert kda.kda_device_error() == (0, 0)


@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (30, 513, 12288), (250, 384, 2048), (1030, 1025, 4112), (2048, 512, 1024)])
def test_against_fp64(M, N, K):
    """Normally distributed rows of uneven size.  A product is exact; each of the K / 32 instructions, and each join of
    partial sums (8 at most), is counted with an error of 2^-22 of the sum of sizes."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M, K, device="cuda", generator=g) * torch.exp(2 * torch.randn(M, 1, device="cuda", generator=g))
    y = torch.randn(N, K, device="cuda", generator=g) * torch.exp(torch.randn(1, K, device="cuda", generator=g))
    (a, sa), (w, sw) = kda.kda_fp8_quant(x, 1), kda.kda_fp8_quant(y, 128)
    da, dw = _dense(a, sa, 1), _dense(w, sw, 128)
    want, size = da @ dw.t(), da.abs() @ dw.abs().t()
    f, h = kda.kda_fp8_matmul(a, sa, w, sw, torch.float32), kda.kda_fp8_matmul(a, sa, w, sw)
    tol = (K / 32 + 8) * 2.0 ** -22 * size
    assert ((f.double() - want).abs() <= tol).all()
    assert ((h.double() - want).abs() <= tol + 2.0 ** -8 * want.abs()).all()
    assert torch.equal(f.bfloat16(), h)


@pytest.mark.parametrize("M", [5, 200, 1300])
def test_values_that_are_not_finite(M):
    """A NaN code or scale of a row of a, or of w: that row, and that block's columns, alone."""
    N, K = 300, 512
    a, sa, w, sw = _exact_operands(M, N, K, 7)
    want = _dense(a.cuda(), sa.cuda(), 1) @ _dense(w.cuda(), sw.cuda(), 128).t()
    a.view(torch.uint8)[3, 100] = 0x7f
    sa[M - 1, 2] = 255
    w.view(torch.uint8)[17, 511] = 0xff
    sw[2, 3] = 255
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[3] = nan[M - 1] = True
    nan[:, 17] = nan[:, 256:] = True
    got = kda.kda_fp8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), torch.float32)
    assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], want.float()[~nan])


@pytest.mark.parametrize("M", [3, 129, 1030])
def test_scales_over_the_range(M):
    """Bytes from 0 to 254 that leave the product in fp32's normal range."""
    N, K = 200, 256
    a, sa, w, sw = _exact_operands(M, N, K, 11)
    for b in (0, 1, 40, 127, 200, 253, 254):
        sa[:], sw[:] = b, 254 - b
        got = kda.kda_fp8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), torch.float32)
        want = (a.double() @ w.double().t()).cuda()   # 2^(b - 127) 2^(127 - b)
        assert torch.equal(got, want.float()), b


@pytest.mark.parametrize("M,N", [(4, 300), (140, 513), (1100, 1000)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides(M, N, dt):
    """Rows cut out of wider ones, the output into columns of another tensor, whose other values stay."""
    K = 336
    a, sa, w, sw = (t.cuda() for t in _exact_operands(M, N, K, 13))
    wide_a = torch.full((M, K + 48), 1.0, device="cuda").to(torch.float8_e4m3fn)
    wide_w = torch.full((N, K + 16), 1.0, device="cuda").to(torch.float8_e4m3fn)
    wide_a[:, 16:16 + K], wide_w[:, :K] = a, w
    t = torch.float32 if dt == "f32" else torch.bfloat16
    want = kda.kda_fp8_matmul(a, sa, w, sw, t)
    for pad, at in ((16, 0), (7, 3), (1, 1), (32, 16)):
        big = torch.full((M, N + pad), -5.0, device="cuda", dtype=t)
        out = big[:, at:at + N]
        got = kda.kda_fp8_matmul(wide_a[:, 16:16 + K], sa, wide_w[:, :K], sw, out=out)
        assert got is out and torch.equal(out, want), (pad, at)
        assert (big[:, :at] == -5).all() and (big[:, at + N:] == -5).all()


def test_no_rows():
    a, sa, w, sw = (t.cuda() for t in _exact_operands(0, 128, 64, 1))
    assert kda.kda_fp8_matmul(a, sa, w, sw).shape == (0, 128)
    a, sa, w, sw = (t.cuda() for t in _exact_operands(3, 0, 64, 1))
    assert kda.kda_fp8_matmul(a, sa, w, sw).shape == (3, 0)


def test_refuses_on_the_gpu():
    a, sa, w, sw = (t.cuda() for t in _exact_operands(4, 256, 128, 1))
    for bad in (lambda: kda.kda_fp8_matmul(a, sa.t(), w, sw), lambda: kda.kda_fp8_matmul(a, sa, w, sw[:1]),
                lambda: kda.kda_fp8_matmul(a, sa, w[:, :112], sw), lambda: kda.kda_fp8_matmul(a, sa, w, sw.cpu()),
                lambda: kda.kda_fp8_matmul(a.t(), sa, w, sw), lambda: kda.kda_fp8_matmul(a, sa, w, sw, out=torch.zeros(4, 255, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(kda.KdaError):
        kda.kda_fp8_matmul(a[:, :120], sa, w[:, :120], sw)    # K not a multiple of 16
    with pytest.raises(kda.KdaError):
        kda.kda_fp8_matmul(a[:, 8:], sa, w[:, 8:], sw)        # begins inside 16 bytes


@pytest.mark.parametrize("M,N", [(70000, 33000), (66000, 32769)])
def test_outputs_beyond_2_31_elements(M, N):
    """Both ends of an output of 2.2e9 values, by tensor stores and by rows that begin anywhere."""
    K = 144
    a, sa, w, sw = (t.cuda() for t in _exact_operands(M, N, K, 3))
    got = kda.kda_fp8_matmul(a, sa, w, sw)
    for rows in (slice(0, 300), slice(M - 300, M)):
        want = _dense(a[rows], sa[rows], 1) @ _dense(w, sw, 128).t()
        assert torch.equal(got[rows], want.bfloat16())


def test_many_rows_of_few_columns():
    """More rows than a grid's second dimension has blocks of 16."""
    M, N, K = 1100000, 24, 32
    a, sa, w, sw = (t.cuda() for t in _exact_operands(M, N, K, 5))
    got = kda.kda_fp8_matmul(a, sa, w, sw)
    assert torch.equal(got, (_dense(a, sa, 1) @ _dense(w, sw, 128).t()).bfloat16())


@pytest.mark.parametrize("pairs", ["0", "1"])
@pytest.mark.parametrize("M,N,K", [(130, 300, 16), (257, 500, 272), (129, 300, 656), (70, 900, 1296)])
def test_scales_at_any_address(M, N, K, pairs, monkeypatch):
    """Scale bytes that begin and end between 32-bit words, with other bytes around them."""
    monkeypatch.setenv("KDA_FP8_PAIR", pairs)
    a, sa, w, sw = (t.cuda() for t in _exact_operands(M, N, K, 7))
    want = kda.kda_fp8_matmul(a, sa, w, sw, torch.float32)
    assert torch.equal(want, (_dense(a, sa, 1) @ _dense(w, sw, 128).t()).float())
    for i in range(1, 8):
        def moved(t, by):
            room = torch.full((t.numel() + 8,), 255, dtype=torch.uint8, device="cuda")
            room[by:by + t.numel()] = t.flatten()
            return room[by:by + t.numel()].view(t.shape)
        assert torch.equal(kda.kda_fp8_matmul(a, moved(sa, i % 4), w, moved(sw, i // 2), torch.float32), want)
