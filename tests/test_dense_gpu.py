"""The dense calls on the GPU against plain forms in fp64: 8-bit storage and read-back,
the residual's addition with its norm, rotary positions."""
import numpy as np
import pytest
import torch

import dense_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.double().cpu().numpy()


def _bytes(codes):
    return codes.view(torch.uint8).cpu().numpy()


def _rows(T, C, dt, seed, wide=False):
    """Values over many powers of two when wide."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C, generator=g, dtype=torch.float64)
    if wide:
        x *= torch.exp2(torch.randint(-40, 40, (T, C), generator=g).double())
    return x.to(DT[dt])


# ------------------------------------------------------------------ 8-bit storage
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("T,C", [(1, 1), (1, 16), (3, 127), (2, 128), (5, 129), (129, 250), (128, 1024), (257, 1032), (300, 77), (2, 5001),
                                 (1, 40000)])
def test_stored_bit_by_bit(T, C, rows, dt):
    x = _rows(T, C, dt, T + C, wide=T % 2 == 1)
    codes, scales = kda.kda_fp8_quant(x.cuda(), rows)
    c, b = ref.stored(_np(x), rows)
    assert np.array_equal(scales.cpu().numpy(), b)
    assert np.array_equal(_bytes(codes), c)
    for out in (torch.float32, torch.bfloat16):
        v = kda.kda_fp8_values(codes, scales, rows, out)
        want = torch.from_numpy(ref.value(c, b, rows)).to(torch.float32).to(out)
        assert torch.equal(v.cpu(), want)
    assert kda.kda_device_error() == (0, 0)


@pytest.mark.parametrize("rows", [1, 128])
def test_edges_of_the_format(rows):
    """Ties, the borders of a scale, subnormals, the largest numbers, and blocks that are not finite."""
    x = np.zeros((130, 300), np.float32)
    x[0, :8] = [448, 17, 19, 21, 2.0 ** -10, 3 * 2.0 ** -10, -17, 0]
    x[1, 0], x[2, 0], x[3, 0], x[4, 0] = 448.00003, 3.4028235e38, 1e-45, -1.17549435e-38
    x[5, 130], x[6, 131], x[7, 299], x[8, 128] = np.inf, np.nan, -np.inf, -0.0
    x[9, :128] = 2.0 ** -126
    x[129, 299] = 7
    codes, scales = kda.kda_fp8_quant(torch.from_numpy(x).cuda(), rows)
    c, b = ref.stored(x, rows)
    assert np.array_equal(scales.cpu().numpy(), b) and np.array_equal(_bytes(codes), c)
    v = kda.kda_fp8_values(codes, scales, rows, torch.float32).cpu()
    assert torch.equal(v, torch.from_numpy(ref.value(c, b, rows)).float()) or \
        np.array_equal(v.numpy(), ref.value(c, b, rows).astype(np.float32), equal_nan=True)
    assert v[0 if rows == 128 else 5, 130].isnan()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("C", [256, 131])
def test_subnormal_bf16(C, rows):
    """Every subnormal bf16 and its neighbours, alone in their blocks and beside larger values."""
    x = torch.arange(0, 512, dtype=torch.int16).view(torch.bfloat16)[:, None].repeat(1, C)
    x[:, 1::2] *= -1
    x[256:, 3] = torch.arange(256).to(torch.bfloat16) * 2.0 ** -120
    codes, scales = kda.kda_fp8_quant(x.cuda(), rows)
    c, b = ref.stored(_np(x), rows)
    assert np.array_equal(scales.cpu().numpy(), b) and np.array_equal(_bytes(codes), c)


def test_every_code_and_scale_byte_reads_back():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 2)
    want = ref.value(codes.numpy(), scales.numpy(), 1)
    for out in (torch.float32, torch.bfloat16):
        v = kda.kda_fp8_values(codes.view(torch.float8_e4m3fn).cuda(), scales.cuda(), 1, out).cpu()
        with np.errstate(over="ignore"):
            w = torch.from_numpy(want.astype(np.float32)).to(out)
        assert torch.equal(v.isnan(), w.isnan()) and torch.equal(v[~v.isnan()], w[~w.isnan()])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
def test_stored_from_strided_rows(dt, rows):
    """Rows cut out of wider ones: aligned, and at odd places."""
    big = _rows(200, 700, dt, 5).cuda()
    for lo, hi in ((0, 256), (64, 512), (3, 300), (1, 257), (8, 690)):
        x = big[:, lo:hi]
        codes, scales = kda.kda_fp8_quant(x, rows)
        c, b = ref.stored(_np(x), rows)
        assert np.array_equal(scales.cpu().numpy(), b) and np.array_equal(_bytes(codes), c), (lo, hi)


# ------------------------------------------------------------------ norm
def _norm_tol(y, dt):
    """The sum of squares: 32 fused steps a thread and 10 additions of positive terms, 2^-24 each, half of it in
    the root; s, the mean, eps, root, quotient and two products, 2^-24 each: 28 in all, 32 counted.  The output's
    own rounding on top."""
    return (32 * 2.0 ** -24 + (2.0 ** -8 if dt == "bf16" else 0)) * np.abs(y) + 2.0 ** -148


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("T,C", [(1, 1), (1, 7), (9, 16), (33, 8), (70, 12), (300, 24), (129, 64), (1000, 100), (65, 128), (41, 127), (6, 129), (5, 256), (3, 257), (17, 512), (64, 1001), (5, 4096), (3, 12288), (2, 16385),
                                 (1, 32768), (4100, 600), (4099, 777), (5000, 513), (4097, 896)])
def test_norm(T, C, add, dt):
    x, r = _rows(T, C, dt, T * C), _rows(T, C, dt, T * C + 1) if add else None
    w = torch.randn(C, generator=torch.Generator().manual_seed(3))
    for weight in (w, None):
        wd = None if weight is None else weight.cuda()
        y, h = kda.kda_add_rmsnorm(x.cuda(), r.cuda() if add else None, wd, 1e-5)
        s, want = ref.norm(_np(x), _np(r) if add else None, None if weight is None else _np(weight), np.float64(np.float32(1e-5)))
        assert (np.abs(_np(y) - want) <= _norm_tol(want, dt)).all()
        codes, scales, h8 = kda.kda_add_rmsnorm_fp8(x.cuda(), r.cuda() if add else None, wd, 1e-5)
        # the scale: that of a largest value within the tolerance; the codes: the nearest to such a value
        near = 1 + 32 * 2.0 ** -24
        b = scales.cpu().numpy()
        lo, hi = ref.scale_bytes(want / near, 1), ref.scale_bytes(want * near, 1)
        assert ((b >= lo) & (b <= hi)).all()
        v = ref.value(_bytes(codes), b, 1)
        unit = np.ldexp(1.0, ref.per_element(b, 1, T, C) - 127)
        step = np.ldexp(1.0, np.maximum(np.frexp(np.abs(want) * near / unit)[1] - 1, -6) - 3) * unit
        assert (np.abs(v - want) <= 0.5 * step + _norm_tol(want, "f32")).all()
        if add:
            sum32 = (x.float() + r.float()).to(DT[dt])
            assert torch.equal(h.cpu(), sum32) and torch.equal(h8.cpu(), sum32)
        else:
            assert h is None and h8 is None
    assert kda.kda_device_error() == (0, 0)


@pytest.mark.parametrize("C", [64, 27, 300, 4096])
def test_norm_range(C):
    """Squares beyond fp32's range and below it, rows of zeros, eps of 0, values that are not finite."""
    x = _rows(8, C, "f32", 9).numpy()
    x[0] *= 1e30
    x[1] *= np.float32(1e-30)
    x[2] = 0
    x[3] = 0
    x[3, C // 2] = 2.0 ** 127
    x[4] *= np.float32(2.0 ** -140)
    x[5] = np.float32(3e38)
    x[6, 3], x[7, 5] = np.inf, np.nan
    for eps in (0.0, 1e-6):
        y, _ = kda.kda_add_rmsnorm(torch.from_numpy(x).cuda(), None, None, eps)
        _, want = ref.norm(x.astype(np.float64), None, None, np.float64(np.float32(eps)))
        y = _np(y)
        got = y[:6] if eps else np.delete(y, 2, 0)[:5]
        want = want[:6] if eps else np.delete(want, 2, 0)[:5]
        assert (np.abs(got - want) <= _norm_tol(want, "f32")).all()
        if not eps:
            assert np.isnan(y[2]).all()                       # 0 / 0
        assert np.isnan(y[6, 3]) and (np.delete(y[6], 3) == 0).all() and np.isnan(y[7]).all()
    codes, scales, _ = kda.kda_add_rmsnorm_fp8(torch.from_numpy(x).cuda(), None, None, 1e-6)
    b = scales.cpu().numpy()
    assert (b[:6] < 255).all() and b[6, 0] == 255 and (b[6, 1:] == 1).all() and (b[7] == 255).all()


@pytest.mark.parametrize("C", [64, 4096])
def test_norm_with_a_large_eps(C):
    """An eps beside squares beyond fp32's range, and one far above them."""
    x = _rows(4, C, "f32", 2).numpy() * np.float32(1e19)
    for eps in (1e30, 1e38, 3e38):
        y, _ = kda.kda_add_rmsnorm(torch.from_numpy(x).cuda(), None, None, eps)
        _, want = ref.norm(x.astype(np.float64), None, None, np.float64(np.float32(eps)))
        assert (np.abs(_np(y) - want) <= _norm_tol(want, "f32")).all()


def test_norm_in_place_and_strided():
    big, res = _rows(33, 700, "bf16", 1).cuda(), _rows(33, 512, "bf16", 2).cuda()
    for lo in (0, 8, 5):
        x = big[:, lo:lo + 512]
        y, h = kda.kda_add_rmsnorm(x, res)
        mine = res.clone()
        y2, h2 = kda.kda_add_rmsnorm(x, mine, residual_out=mine)      # the residual stream, updated
        assert h2 is mine and torch.equal(mine, h) and torch.equal(y, y2)
        c, s, h3 = kda.kda_add_rmsnorm_fp8(x.contiguous(), res)
        mine = x.contiguous()
        c2, s2, _ = kda.kda_add_rmsnorm_fp8(mine, res, residual_out=mine)   # over x
        assert torch.equal(mine, h3) and torch.equal(c.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(s, s2)
    with pytest.raises(ValueError):
        kda.kda_add_rmsnorm(x, res, residual_out=big)
    with pytest.raises(kda.KdaError):
        kda.kda_add_rmsnorm(torch.zeros(1, 32769, device="cuda"))


def test_no_rows_and_no_columns():
    for T, C in ((0, 64), (4, 0)):
        x = torch.zeros(T, C, device="cuda")
        assert kda.kda_add_rmsnorm(x, x)[0].shape == (T, C)
        c, s = kda.kda_fp8_quant(x)
        assert c.shape == (T, C) and kda.kda_fp8_values(c, s).shape == (T, C)
        assert kda.kda_fp8_quant(x, 128)[1].shape == (0, 1) if T == 0 else True


def test_matrices_beyond_2_31_elements():
    """The last rows of 2.2e9 values: norm, 8 bits and back, and the rotation."""
    T, C = 1100000, 2048
    x = torch.zeros(T, C, device="cuda", dtype=torch.bfloat16)
    x[-3:] = _rows(3, C, "bf16", 4).cuda()
    want, _ = kda.kda_add_rmsnorm(x[-3:].contiguous())
    y, h = kda.kda_add_rmsnorm(x, x)
    assert torch.equal(h[-3:], 2 * x[-3:]) and (y[-3:] - want).abs().max() <= 2.0 ** -7 * want.abs().max() and not h[:-3].any()
    del y, h
    for rows in (1, 128):
        codes, scales = kda.kda_fp8_quant(x, rows)
        tail = T - T % 128 if rows == 128 else T - 3
        c, s = kda.kda_fp8_quant(x[tail:], rows)
        assert torch.equal(codes[tail:].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[-s.shape[0]:], s)
        v = kda.kda_fp8_values(codes, scales, rows)
        assert torch.equal(v[tail:], kda.kda_fp8_values(c, s, rows)) and not v[:tail].any()
        del codes, v
    freqs, _ = kda.kda_rotary_freqs(128)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    q = x.view(T, 16, 128)
    yq, _ = kda.kda_rotary(q, None, pos, freqs)
    assert torch.equal(yq[-3:], kda.kda_rotary(q[-3:].contiguous(), None, pos[-3:].contiguous(), freqs)[0]) and not yq[:-3].any()


# ------------------------------------------------------------------ rotary
def _rot_tol(x, want, amp, dt):
    """Each product: the angle to 2^-25 of a turn (2e-7 rad) and sine and cosine to 2^-23, the amplitude, the product and
    the sum 2^-24 each, relative to a pair's size: below 2^-20 of |a| + |b|, counted as twice the largest of the head."""
    size = 2 * np.abs(x).max(-1, keepdims=True) * max(abs(amp), 1.0)
    return 2.0 ** -20 * size + (2.0 ** -8 if dt == "bf16" else 0) * np.abs(want)


CASES = [(1, 1, 1, 64, 64), (7, 6, 2, 128, 128), (33, 3, 1, 128, 64), (5, 2, 2, 96, 96), (9, 2, 1, 50, 30), (4, 1, 0, 8, 2), (300, 12, 4, 64, 16),
         (3, 2, 1, 1024, 1024), (2, 5, 3, 7, 4), (6, 3, 2, 40, 32), (16, 2, 2, 16, 0)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", CASES)
def test_rotary(T, Hq, Hk, D, rot, interleaved, dt):
    q, k = _rows(T * Hq, D, dt, T + D).view(T, Hq, D), _rows(T * Hk, D, dt, T + D + 1).view(T, Hk, D)
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[::3] = torch.randint(0, 5000, (len(pos[::3]),), generator=g, dtype=torch.int64).to(torch.int32)
    if T > 4:
        pos[1], pos[4] = -1, 0
    freqs, _ = kda.kda_rotary_freqs(rot, 500.0, device="cpu")
    for amp, inverse in ((1.0, False), (1.25, True)):
        yq, yk = kda.kda_rotary(q.cuda(), k.cuda() if Hk else None, pos.cuda(), freqs.cuda(), amp, interleaved, inverse)
        for x, y in ((q, yq), (k, yk))[:2 if Hk else 1]:
            want = ref.rotate(_np(x), pos.numpy(), freqs.numpy(), amp, interleaved, inverse)
            assert (np.abs(_np(y) - want) <= _rot_tol(_np(x), want, amp, dt)).all()
            still = torch.from_numpy(pos.numpy() < 0)
            assert torch.equal(y.cpu()[still], x[still]) and torch.equal(y.cpu()[..., rot:], x[..., rot:])
    assert kda.kda_device_error() == (0, 0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot,extra", [(64, 64, 0), (128, 32, 0), (64, 48, 5), (20, 10, 3)])
def test_rotary_in_place_and_strided(D, rot, extra, dt):
    """Queries and keys as parts of one projection's rows, turned where they lie; the rest of the rows stays."""
    T, Hq, Hk = 37, 6, 2
    width = (Hq + 2 * Hk) * D + extra
    p = _rows(T, width, dt, 4).cuda()
    q, k = p[:, :Hq * D].unflatten(1, (Hq, D)), p[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000 - 2000
    freqs, amp = kda.kda_rotary_freqs(rot, 10000.0, "ramp", 8.0, 4096)
    yq, yk = kda.kda_rotary(q, k, pos, freqs, amp)
    assert yq.is_contiguous() and yk.is_contiguous()
    before = p.clone()
    a, b = kda.kda_rotary(q, k, pos, freqs, amp, q_out=q, k_out=k)
    assert a is q and b is k and torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(p[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])
    heads_first = torch.empty(Hq, T, D, dtype=DT[dt], device="cuda")     # another order of the output
    kda.kda_rotary(before[:, :Hq * D].unflatten(1, (Hq, D)), None, pos, freqs, amp, q_out=heads_first.transpose(0, 1))
    assert torch.equal(heads_first.transpose(0, 1), yq)
    with pytest.raises(kda.KdaError):
        kda.kda_rotary(q, k, pos, freqs, q_out=p[:, D:(Hq + 1) * D].unflatten(1, (Hq, D)))


@pytest.mark.parametrize("T", [1, 2, 37])
@pytest.mark.parametrize("order", ["tokens", "heads", "heads and more", "apart"])
def test_rotary_one_part_in_place(T, order):
    """Queries where they lie with keys between their tokens or heads, into new memory and in place."""
    H, D = 4, 64
    p = _rows(T, 2 * H * D + 64, "bf16", T).cuda()
    if order == "tokens":
        q, k = p[:, :H * D].unflatten(1, (H, D)), p[:, H * D:(H + 2) * D].unflatten(1, (2, D))
    elif order == "heads":
        both = p[:, :2 * H * D].contiguous().view(T, 2 * H, D)
        q, k = both[:, 0::2], both[:, 1::2]
    elif order == "heads and more":   # the head stride does not divide the tokens', but the tokens do not reach one another
        both = p[:, :2 * H * D].unflatten(1, (2 * H, D))
        q, k = both[:, :H], both[:, H:]
    else:
        q, k = p[:, :H * D].contiguous().view(T, H, D), p[:, H * D:2 * H * D].contiguous().view(T, H, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 991 - 1
    freqs, _ = kda.kda_rotary_freqs(D)
    yq, yk = kda.kda_rotary(q, k, pos, freqs)
    keys = k.clone()
    a, b = kda.kda_rotary(q, k, pos, freqs, q_out=q)
    assert a is q and torch.equal(q, yq) and torch.equal(b, yk) and torch.equal(k, keys)
    queries = q.clone()
    kda.kda_rotary(q, k, pos, freqs, k_out=k)
    assert torch.equal(q, queries) and torch.equal(k, yk)
    with pytest.raises(kda.KdaError):
        kda.kda_rotary(q, q, pos, freqs, q_out=q, k_out=q)
    with pytest.raises(kda.KdaError):
        kda.kda_rotary(q, q[:, 1:], pos, freqs, q_out=q)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_is_the_gradient(interleaved):
    """The rotation is linear: <inverse(g), x> = <g, rotation(x)> for any x, the gradient by its definition."""
    T, H, D = 11, 3, 64
    x, g = (_rows(T * H, D, "f32", s).view(T, H, D).cuda() for s in (1, 2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 777
    freqs, _ = kda.kda_rotary_freqs(48)
    y, _ = kda.kda_rotary(x, None, pos, freqs, 1.5, interleaved)
    dx, _ = kda.kda_rotary(g, None, pos, freqs, 1.5, interleaved, inverse=True)
    both = (dx.double() * x.double()).sum() - (g.double() * y.double()).sum()
    assert abs(both) <= 2.0 ** -20 * 1.5 * 2 * (x.double().abs() * g.double().abs().flip(-1).amax(-1, keepdim=True)).sum()
    back, _ = kda.kda_rotary(kda.kda_rotary(x, None, pos, freqs, 1.0, interleaved)[0], None, pos, freqs, 1.0, interleaved, inverse=True)
    assert (back - x).abs().max() <= 2.0 ** -18 * x.abs().max()


def test_rotary_far_positions_of_fast_pairs():
    """Angles of 2^31 radians, and a frequency of several turns a token."""
    freqs = torch.tensor([1.0, 0.999999999, 6.5, 100.0, 1e-9, 3.0])
    freqs = freqs.double()
    pos = torch.tensor([2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30 + 7, 123456789], dtype=torch.int32)
    x = _rows(4 * 2, 12, "f32", 8).view(4, 2, 12)
    y, _ = kda.kda_rotary(x.cuda(), None, pos.cuda(), freqs.cuda())
    want = ref.rotate(_np(x), pos.numpy(), freqs.numpy(), 1.0, False, False)
    assert (np.abs(_np(y) - want) <= _rot_tol(_np(x), want, 1.0, "f32")).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(9731, 1, 1, 64, 64), (20000, 2, 1, 64, 32), (10007, 1, 0, 6, 4), (40001, 4, 2, 128, 128),
                                             (20000, 12, 1, 64, 64), (9000, 8, 8, 128, 64), (15001, 9, 3, 20, 12)])
def test_rotary_many_tokens(T, Hq, Hk, D, rot, interleaved, dt):
    """Few heads and more tokens than the chip holds warps, the formula in fp64 on the GPU (angles below 2^31 * 1e-4, so
    that fp64's own error in them stays below 2^-30)."""
    x = _rows(T * (Hq + Hk), D, dt, T).view(T, Hq + Hk, D).cuda()
    q, k = x[:, :Hq], x[:, Hq:] if Hk else None
    pos = torch.randint(-1000, 2 ** 31 - 1, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
    pos[5::7] = -1
    freqs, _ = kda.kda_rotary_freqs(rot, 100.0)
    freqs = freqs * 1e-4
    yq, yk = kda.kda_rotary(q, k, pos, freqs, 1.0, interleaved)
    y = yq if yk is None else torch.cat([yq, yk], 1)
    ang = (pos.double()[:, None] * freqs)[:, None]
    still = (pos < 0)[:, None, None]
    c, s = torch.where(still, 1.0, ang.cos()), torch.where(still, 0.0, ang.sin())
    want = x.double().clone()
    i = 2 * torch.arange(rot // 2, device="cuda") if interleaved else torch.arange(rot // 2, device="cuda")
    j = i + 1 if interleaved else i + rot // 2
    want[..., i], want[..., j] = x.double()[..., i] * c - x.double()[..., j] * s, x.double()[..., i] * s + x.double()[..., j] * c
    size = 2 * x.double().abs().amax(-1, keepdim=True)
    assert ((y.double() - want).abs() <= 2.0 ** -20 * size + (2.0 ** -8 if dt == "bf16" else 0) * want.abs()).all()
    assert torch.equal(y[pos < 0], x[pos < 0])


def test_rotary_many_heads_at_any_alignment():
    """66,560 single pairs a token, more tokens than warps: each as in a call of its own."""
    T, H, D = 4900, 1024, 130
    x = torch.randn(T, H * D + 1, device="cuda").bfloat16()[:, 1:].unflatten(1, (H, D))
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    freqs, _ = kda.kda_rotary_freqs(D)
    yq, yk = kda.kda_rotary(x[:, :1000], x[:, 1000:], pos, freqs)
    for t in (0, 1, 2500, T - 1):
        want, _ = kda.kda_rotary(x[t:t + 1, 3:].contiguous(), None, pos[t:t + 1].contiguous(), freqs)
        assert torch.equal(torch.cat([yq[t:t + 1, 3:], yk[t:t + 1]], 1), want)
    want = ref.rotate(_np(x[-1:, -2:]), pos[-1:].cpu().numpy(), freqs.cpu().numpy(), 1.0, False, False)
    assert (np.abs(_np(yk[-1:, -2:]) - want) <= _rot_tol(_np(x[-1:, -2:]), want, 1.0, "bf16")).all()


def test_rotary_no_tokens():
    q = torch.zeros(0, 4, 64, device="cuda")
    y, _ = kda.kda_rotary(q, None, torch.zeros(0, dtype=torch.int32, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda"))
    assert y.shape == q.shape
