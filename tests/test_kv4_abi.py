"""The 4-bit cache's calls without a GPU: refusals of bad arguments on the host,
in the C ABI and in the Python binding, and the plain forms that the GPU tests
compare with."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda
from linear_attention_recurrence_chunk_gb300 import kv4

G = 1 << 30
FAKE = 1 << 44   # never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    return kv4._lib()


def test_cache_bytes(lib):
    f = lib.kda_kv4_cache_bytes
    bad = (1 << 64) - 1
    assert f(10, 8, 64, 128) == 10 * 8 * 4 * 17 * 128
    assert f(3, 2, 16, 64) == 3 * 2 * 17 * 64
    assert f(0, 8, 64, 128) == 0
    for args in [(10, 8, 64, 96), (10, 8, 40, 128), (10, 8, 0, 128), (10, 8, 8192, 128), (10, 0, 64, 128),
                 (-1, 8, 64, 128), ((1 << 31) // 64, 8, 64, 128)]:
        assert f(*args) == bad, args


def _map(lib, **kw):
    a = dict(cached=FAKE, new=FAKE + G, N=4, table=FAKE + 2 * G, mp=8, free=FAKE + 3 * G, F=100, start=FAKE + 4 * G,
             ps=64, T=100, cu=FAKE + 5 * G, lens=FAKE + 6 * G, slots=FAKE + 7 * G, pos=FAKE + 8 * G, nxt=FAKE + 9 * G)
    a.update(kw)
    return lib.kda_page_map(a["cached"], a["new"], a["N"], a["table"], a["mp"], a["free"], a["F"], a["start"], a["ps"],
                            a["T"], a["cu"], a["lens"], a["slots"], a["pos"], a["nxt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(cached=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(free=None), 1), (dict(start=None), 1),
    (dict(cu=None), 1), (dict(lens=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(nxt=None), 1),
    (dict(N=-1), 1), (dict(mp=-1), 1), (dict(F=-1), 1), (dict(T=-1), 1), (dict(ps=40), 1), (dict(ps=0), 1),
    (dict(ps=8192), 1), (dict(N=28673), 2), (dict(slots=FAKE + 7 * G + 4), 1), (dict(pos=FAKE + 8 * G + 8), 1),
    (dict(cached=FAKE + 2), 1), (dict(cu=FAKE + 4), 1),           # cu over cached_lens
    (dict(nxt=FAKE + 4 * G), 1),                                   # free_next over free_start
    (dict(table=FAKE + 3 * G), 1), (dict(pos=FAKE + 7 * G + 16), 1), (dict(T=(1 << 31)), 1)])
def test_page_map_refusals(lib, kw, want):
    assert _map(lib, **kw) == want


def _append(lib, **kw):
    a = dict(k=FAKE, v=FAKE + 8 * G, slots=FAKE + 16 * G, T=100, H=8, D=128, kt=1024, kh=128, vt=1024, vh=128, dt=1,
             cache=FAKE + 32 * G, pages=10, ps=64)
    a.update(kw)
    return lib.kda_kv4_append(a["k"], a["v"], a["slots"], a["T"], a["H"], a["D"], a["kt"], a["kh"], a["vt"], a["vh"],
                              a["dt"], a["cache"], a["pages"], a["ps"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(cache=None), 1), (dict(dt=7), 1), (dict(T=-1), 1),
    (dict(D=96), 2), (dict(H=0), 1), (dict(ps=24), 1), (dict(k=FAKE + 8), 1), (dict(kt=1020), 1), (dict(vh=132), 1),
    (dict(kt=-1024), 1), (dict(cache=FAKE + 32 * G + 8), 1), (dict(cache=FAKE + 64), 1), (dict(slots=FAKE + 16 * G + 2), 1),
    (dict(pages=1 << 30), 1)])
def test_append_refusals(lib, kw, want):
    assert _append(lib, **kw) == want
    assert _append(lib, T=0, k=None, v=None) == 0


def _gather(lib, **kw):
    a = dict(cache=FAKE, pages=10, ps=64, slots=FAKE + G, T=100, H=8, D=128, dt=1, k=FAKE + 2 * G, v=FAKE + 3 * G)
    a.update(kw)
    return lib.kda_kv4_gather(a["cache"], a["pages"], a["ps"], a["slots"], a["T"], a["H"], a["D"], a["dt"], a["k"], a["v"],
                              None)


@pytest.mark.parametrize("kw,want", [
    (dict(cache=None), 1), (dict(slots=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(dt=2), 1), (dict(D=32), 2),
    (dict(k=FAKE + 2 * G + 8), 1), (dict(k=FAKE), 1), (dict(v=FAKE + 2 * G + 64), 1), (dict(T=-5), 1), (dict(ps=17), 1)])
def test_gather_refusals(lib, kw, want):
    assert _gather(lib, **kw) == want
    assert _gather(lib, T=0) == 0


def test_python_binding_refuses():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_page_map(i, i, torch.zeros(4, 8, dtype=torch.int32), i, i[:1], 64, 10)          # not on a GPU
    with pytest.raises(TypeError):
        kda.kda_page_map(i.long(), i, torch.zeros(4, 8, dtype=torch.int32), i, i[:1], 64, 10)   # int64 lengths
    with pytest.raises(ValueError):
        kda.kda_kv4_gather(torch.zeros(2, 1, 4, 17 * 128, dtype=torch.uint8), i)                 # cache not on a GPU
    with pytest.raises(ValueError):
        kda.kda_kv4_gather(torch.zeros(2, 1, 4, 2170, dtype=torch.uint8), i)
    with pytest.raises(kda.KdaError):
        kda.kda_kv4_cache(4, 1, 24, 128, device="cpu")
    assert kda.kda_kv4_cache(4, 2, 32, 64, device="cpu").shape == (4, 2, 2, 17 * 64)


def test_stored_values_of_known_numbers():
    """A group whose scale is 1 (largest |x| 6): every level, every tie, both signs."""
    x = np.array([0, 0.25, 0.26, 0.5, 0.74, 0.75, 1, 1.25, 1.26, 1.5, 1.75, 1.74, 2, 2.5, 2.51, 3, 3.5, 3.49, 4, 5, 5.01, 6,
                  -0.25, -0.75, -1.25, -5, -6, -3.5, 0, 0, 0, 0])
    want = [0, 0, 0.5, 0.5, 0.5, 1, 1, 1, 1.5, 1.5, 2, 1.5, 2, 2, 3, 3, 4, 3, 4, 4, 6, 6, 0, -1, -1, -4, -6, -4, 0, 0, 0, 0]
    c, b = ref.stored(x)
    assert b.tolist() == [127]
    assert ref.value(c, b).tolist() == want
    for top, byte in [(6.0, 127), (6.0001, 128), (3.0, 126), (3.0001, 127), (12.0, 128), (0.0, 1), (2.0 ** -126, 1),
                      (6 * 2.0 ** -126, 1), (6.1 * 2.0 ** -126, 2), (3e38, 253), (np.inf, 255), (np.nan, 255)]:
        y = np.zeros(32)
        y[5] = -top
        assert ref.stored(y)[1].tolist() == [byte], top


def test_unit_layout_round_trip():
    """The byte layout is one-to-one: each nibble and scale byte of a unit is used once."""
    rng = np.random.default_rng(1)
    for D in (64, 128):
        kc, vc = rng.integers(0, 16, (16, D)).astype(np.uint8), rng.integers(0, 16, (16, D)).astype(np.uint8)
        full = np.full((16, D), 15, np.uint8)
        ones = np.full((16, D // 32), 255, np.uint8)
        assert (ref.unit_bytes(full, ones, full, ones) == 255).all()
        zero = np.zeros_like(kc)
        a = ref.unit_bytes(kc, 0 * ones, zero, 0 * ones)
        b = ref.unit_bytes(zero, 0 * ones, vc, 0 * ones)
        assert not a[8 * D:].any() and not b[:8 * D].any()


def test_page_map_reference():
    t, cu, lens, slots, pos, nxt = ref.page_map([3, 0, 16], [2, 17, 0], np.full((3, 3), -1), [5, 6, 7, 8], 1, 16, 20)
    # request 0: page 0 of its row is given as -1, so its tokens have no page
    assert slots.tolist()[:2] == [-1, -1] and pos.tolist()[:2] == [3, 4]
    assert t[1].tolist() == [6, 7, -1] and slots.tolist()[2:] == [6 * 16 + i for i in range(16)] + [7 * 16] + [-1]
    assert cu.tolist() == [0, 2, 19, 19] and lens.tolist() == [5, 17, 16] and nxt == 3


def _attn(lib, **kw):
    a = dict(q=FAKE, qt=1024, qh=128, cache=FAKE + 8 * G, pages=10, ps=64, table=FAKE + 9 * G, mp=4, lens=FAKE + 10 * G,
             cu=None, T=3, N=3, Hq=8, Hkv=2, D=128, mq=1, scale=0.1, dt=1, o=FAKE + 11 * G, lse=None, ws=FAKE + 12 * G,
             wsb=1 << 33)
    a.update(kw)
    return lib.kda_kv4_attention(a["q"], a["qt"], a["qh"], a["cache"], a["pages"], a["ps"], a["table"], a["mp"], a["lens"],
                                 a["cu"], a["T"], a["N"], a["Hq"], a["Hkv"], a["D"], a["mq"], a["scale"], a["dt"], a["o"],
                                 a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(o=None), 1),
    (dict(ws=None), 1), (dict(wsb=100), 1), (dict(ws=FAKE + 12 * G + 128), 1), (dict(dt=3), 1), (dict(D=96), 2),
    (dict(Hq=7), 1), (dict(Hq=258), 2), (dict(Hq=0), 1), (dict(T=4), 1), (dict(mq=2), 1), (dict(mq=0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(ps=20), 1), (dict(mp=-1), 1),
    (dict(N=65536, T=65536), 2), (dict(q=FAKE + 2), 1), (dict(qt=1025), 1), (dict(o=FAKE), 1),
    (dict(lse=FAKE + 11 * G + 16), 1), (dict(o=FAKE + 8 * G + 64), 1), (dict(lens=FAKE + 10 * G + 1), 1),
    (dict(cu=FAKE + 13 * G + 2, mq=3), 1), (dict(N=-1), 1), (dict(T=-1), 1)])
def test_attention_refusals(lib, kw, want):
    assert _attn(lib, **kw) == want
    assert _attn(lib, T=0, N=0, q=None) == 0


def test_attention_workspace(lib):
    f = lib.kda_kv4_attention_workspace_size
    assert 0 < f(3, 3, 8, 2, 128, 1, 1) < f(3, 3, 32, 2, 128, 1, 1) < 1 << 30
    for args in [(3, 3, 7, 2, 128, 1, 1), (3, 3, 8, 2, 100, 1, 1), (3, 3, 8, 2, 128, 0, 1), (-1, 3, 8, 2, 128, 1, 1),
                 (3, 3, 8, 2, 128, 1, 9)]:
        assert f(*args) == (1 << 64) - 1, args
