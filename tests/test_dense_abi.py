"""The dense calls without a GPU: refusals of bad arguments on the host, in the C ABI
and in the Python binding, and the plain forms that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import dense_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda
from linear_attention_recurrence_chunk_gb300 import dense

G = 1 << 34
FAKE = 1 << 44   # never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    return dense._lib()


def _quant(lib, **kw):
    a = dict(x=FAKE, xs=512, T=100, C=512, rows=1, dt=1, codes=FAKE + G, scales=FAKE + 2 * G)
    a.update(kw)
    return lib.kda_fp8_quant(a["x"], a["xs"], a["T"], a["C"], a["rows"], a["dt"], a["codes"], a["scales"], None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(codes=None), dict(scales=None), dict(dt=2), dict(T=-1), dict(C=-1), dict(rows=2), dict(rows=0), dict(xs=511),
    dict(x=FAKE + 1), dict(x=FAKE + 2, dt=0), dict(codes=FAKE + 1000), dict(scales=FAKE + G + 51199), dict(scales=FAKE + 51200),
    dict(T=1 << 31), dict(C=1 << 31), dict(xs=-512), dict(T=1 << 30, C=1 << 30, xs=1 << 30)])
def test_quant_refusals(lib, kw):
    assert _quant(lib, **kw) == 1
    assert _quant(lib, T=0, x=None) == 0 and _quant(lib, C=0, codes=None) == 0


def _values(lib, **kw):
    a = dict(codes=FAKE, scales=FAKE + G, T=100, C=512, rows=128, dt=1, y=FAKE + 2 * G)
    a.update(kw)
    return lib.kda_fp8_values(a["codes"], a["scales"], a["T"], a["C"], a["rows"], a["dt"], a["y"], None)


@pytest.mark.parametrize("kw", [
    dict(codes=None), dict(scales=None), dict(y=None), dict(dt=5), dict(T=-1), dict(rows=64), dict(y=FAKE), dict(y=FAKE + G),
    dict(y=FAKE + 2 * G + 1), dict(C=1 << 31)])
def test_values_refusals(lib, kw):
    assert _values(lib, **kw) == 1
    assert _values(lib, T=0) == 0


def _norm(lib, **kw):
    a = dict(x=FAKE, xs=512, r=FAKE + G, rs=512, w=FAKE + 2 * G, eps=1e-6, T=100, C=512, dt=1, h=FAKE + 3 * G, y=FAKE + 4 * G, codes=None,
             scales=None)
    a.update(kw)
    return lib.kda_add_rmsnorm(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["eps"], a["T"], a["C"], a["dt"], a["h"], a["y"], a["codes"],
                               a["scales"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), 1), (dict(h=None), 1), (dict(r=None), 1), (dict(y=None), 1), (dict(codes=FAKE + 5 * G), 1),
    (dict(y=None, codes=FAKE + 5 * G), 1), (dict(y=None, scales=FAKE + 5 * G), 1), (dict(dt=3), 1), (dict(eps=-1.0), 1),
    (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(C=32769, xs=32769, rs=32769), 2), (dict(xs=500), 1), (dict(rs=100), 1),
    (dict(x=FAKE + 1), 1), (dict(w=FAKE + 2 * G + 2), 1), (dict(h=FAKE + 64), 1), (dict(h=FAKE, xs=1024), 1),
    (dict(h=FAKE + G, rs=520), 1), (dict(y=FAKE + G), 1), (dict(y=FAKE + 3 * G + 512), 1), (dict(y=FAKE + 1024), 1),
    (dict(h=FAKE, y=FAKE), 1), (dict(y=FAKE + 2 * G), 1), (dict(h=FAKE + 2 * G), 1), (dict(T=-1), 1),
    (dict(y=None, codes=FAKE, scales=FAKE + 5 * G), 1), (dict(y=None, codes=FAKE + 5 * G, scales=FAKE + 5 * G + 100), 1),
    (dict(y=None, codes=FAKE + 3 * G + 5, scales=FAKE + 5 * G), 1)])
def test_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want
    assert _norm(lib, T=0, x=None, h=None) == 0


def _matmul(lib, **kw):
    a = dict(a=FAKE, lda=512, sa=FAKE + G, w=FAKE + 2 * G, ldw=512, sw=FAKE + 3 * G, M=10, N=300, K=512, dt=1, out=FAKE + 4 * G, ldo=300)
    a.update(kw)
    return lib.kda_fp8_matmul(a["a"], a["lda"], a["sa"], a["w"], a["ldw"], a["sw"], a["M"], a["N"], a["K"], a["dt"], a["out"], a["ldo"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), 1), (dict(sa=None), 1), (dict(w=None), 1), (dict(sw=None), 1), (dict(out=None), 1), (dict(dt=9), 1), (dict(M=-1), 1),
    (dict(N=-1), 1), (dict(K=0), 1), (dict(K=-16), 1), (dict(K=500, lda=512), 2), (dict(M=1 << 31), 2), (dict(N=1 << 31), 2), (dict(K=(1 << 27) + 16, lda=1 << 28, ldw=1 << 28), 2),
    (dict(lda=496), 1), (dict(lda=520), 1), (dict(ldw=504), 1), (dict(a=FAKE + 8), 1), (dict(w=FAKE + 2 * G + 4), 1),
    (dict(out=FAKE + 4 * G + 1), 1), (dict(out=FAKE + 4 * G + 2, dt=0), 1), (dict(ldo=299), 1), (dict(out=FAKE), 1),
    (dict(out=FAKE + G + 8), 1), (dict(out=FAKE + 2 * G), 1), (dict(out=FAKE + 3 * G), 1), (dict(lda=-512), 1),
    (dict(ldw=1 << 38), 1), (dict(ldo=1 << 38), 1)])
def test_matmul_refusals(lib, kw, want):
    assert _matmul(lib, **kw) == want
    assert _matmul(lib, M=0, a=None) == 0 and _matmul(lib, N=0, w=None) == 0


def _rotary(lib, **kw):
    a = dict(q=FAKE, qt=1280, qh=128, Hq=8, k=FAKE + 2048, kt=1280, kh=128, Hk=2, pos=FAKE + G, T=50, D=128, rot=64, freqs=FAKE + 2 * G, amp=1.0,
             flags=0, dt=1, qo=FAKE + 3 * G, qot=1024, qoh=128, ko=FAKE + 4 * G, kot=256, koh=128)
    a.update(kw)
    return lib.kda_rotary(*(a[n] for n in ("q", "qt", "qh", "Hq", "k", "kt", "kh", "Hk", "pos", "T", "D", "rot", "freqs", "amp", "flags", "dt",
                                           "qo", "qot", "qoh", "ko", "kot", "koh")), None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(freqs=None), 1), (dict(dt=4), 1),
    (dict(T=-1), 1), (dict(D=0), 1), (dict(rot=63), 1), (dict(rot=130), 1), (dict(rot=-2), 1), (dict(flags=4), 1), (dict(amp=math.inf), 1),
    (dict(amp=math.nan), 1), (dict(D=1026), 2), (dict(Hq=1025), 2), (dict(Hq=1000, Hk=100), 2), (dict(Hq=-1), 1), (dict(pos=FAKE + G + 2), 1),
    (dict(freqs=FAKE + 2 * G + 4), 1), (dict(q=FAKE + 1), 1), (dict(qoh=64), 1), (dict(qot=100), 1), (dict(qt=-1280), 1),
    (dict(qo=FAKE), 1),                                     # over its input, with other strides
    (dict(qo=FAKE + 256, qot=1280), 1),                     # shifted by a head
    (dict(qo=FAKE + 4 * G), 1),                             # over k_out
    (dict(qot=128, qoh=128), 1), (dict(qot=512), 1), (dict(kot=128), 1),   # tokens over the heads of others
    (dict(qot=1 << 38), 1),
    (dict(ko=FAKE + 2048), 1), (dict(ko=FAKE + G), 1), (dict(qo=FAKE + 2 * G), 1)])
def test_rotary_refusals(lib, kw, want):
    assert _rotary(lib, **kw) == want
    assert _rotary(lib, T=0, q=None) == 0 and _rotary(lib, Hq=0, Hk=0, q=None, k=None) == 0


_IN = dict(qo=FAKE, qot=1280, qoh=128)   # the queries in place


@pytest.mark.parametrize("kw", [
    dict(k=FAKE, kt=1280, kh=128, Hk=8), dict(k=FAKE + 2046), dict(k=FAKE + 256), dict(k=FAKE + 2560 - 256 + 2),   # keys over the queries
    dict(k=FAKE + 2560 * 7 + 512), dict(k=FAKE + 2560 * 7 - 256), dict(k=FAKE + 2048, kt=640),                # rows on; another stride
    dict(k=FAKE, ko=FAKE, kt=1280, kot=1280), dict(k=FAKE, T=1), dict(k=FAKE + 2 * 128 * 7, T=1, Hk=1),
    dict(k=FAKE + 128, qt=2048, qh=256, qot=2048, qoh=256, kt=2048, kh=256, Hk=8),                            # half a head on
    dict(k=FAKE + 256, qt=2100, qh=256, qot=2100, qoh=256, kt=2100, kh=256, Hk=8)])                           # head steps that miss the tokens'
def test_rotary_in_place_over_the_other_part(lib, kw):
    """What one part reads while the other is turned where it lies."""
    assert _rotary(lib, **{**_IN, **kw}) == 1


def test_python_binding_refuses():
    x = torch.zeros(4, 256)
    c, s = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8)
    for call in (lambda: kda.kda_fp8_quant(x), lambda: kda.kda_fp8_values(c, s), lambda: kda.kda_add_rmsnorm(x),
                 lambda: kda.kda_add_rmsnorm_fp8(x), lambda: kda.kda_fp8_matmul(c, s, c, s[:1]),
                 lambda: kda.kda_rotary(x[None], None, torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.float64))):
        with pytest.raises(ValueError):   # not on a GPU
            call()
    with pytest.raises(TypeError):
        kda.kda_fp8_values(x, s)
    with pytest.raises(TypeError):
        kda.kda_fp8_matmul(x, s, c, s)


def test_levels():
    """Every finite E4M3 value, against PyTorch's type."""
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = ref.value(np.arange(256, dtype=np.uint8)[None], np.full((1, 2), 127, np.uint8), 1)[0]
    assert np.array_equal(got, v, equal_nan=True) and np.isnan(v[127]) and v[126] == 448


def test_stored_values_of_known_numbers():
    for top, byte in [(448.0, 127), (448.1, 128), (224.0, 126), (224.01, 127), (0.0, 1), (2.0 ** -126, 1), (448 * 2.0 ** -126, 1),
                      (449 * 2.0 ** -126, 2), (3e38, 247), (np.inf, 255), (np.nan, 255)]:
        x = np.zeros((1, 130))
        x[0, 5] = -top
        assert ref.stored(x, 1)[1].tolist() == [[byte, 1]], top
    x = np.array([[448, 17, 17.5, 18, 19, 21, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -1.0625, 1.1875]])   # scale 1: ties to the even code
    c, b = ref.stored(x, 1)
    assert ref.value(c, b, 1)[0].tolist() == [448, 16, 18, 18, 20, 20, 2.0 ** -9, 0, 2.0 ** -8, -1, 1.25]


def test_stored_as_torch_rounds():
    """Codes of a block whose scale is 1 are PyTorch's."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 128)).astype(np.float32) * np.exp(rng.standard_normal((64, 128)) * 3).astype(np.float32)
    x = np.clip(x, -448, 448)
    x[:, 0] = 448
    c, b = ref.stored(x, 1)
    assert (b == 127).all()
    assert np.array_equal(c, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_rotary_freqs():
    f, amp = kda.kda_rotary_freqs(8, 100.0, device="cpu")
    assert amp == 1.0 and f.tolist() == [100.0 ** (-i / 4) for i in range(4)]
    assert torch.equal(kda.kda_rotary_freqs(8, 100.0, "linear", 4.0, device="cpu")[0], f / 4)
    g = kda.kda_rotary_freqs(8, 100.0, "base", 4.0, device="cpu")[0]
    assert g[0] == f[0] and abs(g[3] / f[3] - 0.25) < 1e-12
    g, amp = kda.kda_rotary_freqs(128, 10000.0, "ramp", 16.0, 8192, device="cpu")
    h = kda.kda_rotary_freqs(128, 10000.0, device="cpu")[0]
    turns = 8192 * h / (2 * math.pi)
    assert abs(amp - (0.1 * math.log(16) + 1)) < 1e-15
    assert torch.equal(g[turns >= 32], h[turns >= 32]) and torch.allclose(g[turns <= 1], h[turns <= 1] / 16, rtol=1e-12)
    between = (turns < 32) & (turns > 1)
    assert ((g < h) & (g > h / 16))[between].all()
    for bad in (dict(rot=7), dict(base=1.0), dict(factor=0.5), dict(scaling="other"), dict(scaling="ramp"),
                dict(scaling="ramp", original_len=10, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            kda.kda_rotary_freqs(**{"rot": 8, "device": "cpu", **bad})
    assert kda.kda_rotary_freqs(0, device="cpu")[0].numel() == 0
    assert kda.kda_rotary_freqs(2, scaling="base", factor=4.0, device="cpu")[0].tolist() == [1.0]
