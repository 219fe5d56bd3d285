"""How the 8-bit product is cut, without a GPU: the choice by sizes, and refusals of cuts that there are not."""
import ctypes
import random

import pytest

import dense_testutil as ref

G = 1 << 34
FAKE = 1 << 44   # never dereferenced: every case fails validation first


def _fits(M, N, cut):
    rows, split, _ = cut
    return rows == 0 or (-(-M // rows) <= 65535 and -(-N // 128) * -(-M // rows) * split <= 2 ** 31 - 1)


@pytest.mark.parametrize("sms", [132, 148, 152, 160])
def test_every_choice_is_a_cut(sms):
    rng = random.Random(sms)
    for _ in range(2000):
        M, N, K = int(2 ** rng.uniform(0, 24)), int(2 ** rng.uniform(0, 20)), 16 * int(2 ** rng.uniform(0, 12))
        for dt in (0, 1):
            rows, split, deep = ref.choice(M, N, K, dt, sms)
            assert (rows, split) == (0, 1) or (rows in (16, 32, 64, 128, 256) and split in (1, 2, 4, 8) and split <= -(-K // 512))
            assert _fits(M, N, (rows, split, deep))


@pytest.mark.parametrize("M,N,K", [(65535 * 256 + 1, 1, 16), (65535 * 16 + 1, 24, 32), (2 ** 31 - 512, 1, 16), (1, 2 ** 31 - 512, 16)])
def test_choices_at_a_grids_limits(M, N, K):
    for dt in (0, 1):
        assert _fits(M, N, ref.choice(M, N, K, dt))


@pytest.mark.parametrize("sms", [148, 152])
def test_parts_of_k_do_not_depend_on_the_output_type(sms):
    """They set the order of the sums."""
    rng = random.Random(3)
    sizes = [(39, 6169, 7184), (55, 4345, 6448), (61, 4955, 9888)]
    sizes += [(int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(4, 14)), 16 * int(2 ** rng.uniform(2, 10))) for _ in range(5000)]
    for size in sizes:
        assert ref.choice(*size, 0, sms)[1] == ref.choice(*size, 1, sms)[1], size


@pytest.mark.parametrize("bad", [dict(M=0), dict(N=0), dict(K=15), dict(dt=2), dict(sms=1), dict(M=2 ** 31), dict(cut=None)])
def test_choice_refuses(bad):
    a = dict(M=10, N=20, K=512, dt=1, sms=152, cut=(ctypes.c_int32 * 3)())
    a.update(bad)
    assert ref.cut_library().kda_fp8_matmul_choice(a["M"], a["N"], a["K"], a["dt"], a["sms"], a["cut"]) == 1


@pytest.mark.parametrize("M,cut,want", [
    (100, (8, 1, 1), 1), (100, (24, 1, 1), 1), (100, (512, 1, 1), 1), (100, (-16, 1, 1), 1), (100, (16, 3, 1), 1), (100, (16, 0, 1), 1),
    (100, (16, 16, 1), 1), (100, (16, 4, 1), 1), (100, (0, 2, 1), 1),               # K has two groups of four blocks
    (65535 * 16 + 1, (16, 1, 0), 2), (65535 * 256 + 1, (256, 1, 1), 2), (100, (16, 1, 1), 1)])
def test_cuts_that_there_are_not(M, cut, want):
    """(The last one is a cut, of a call with an operand that is missing.)"""
    N, K = 300, 1024
    w = None if cut == (16, 1, 1) else FAKE + G
    lib = ref.cut_library()
    assert lib.kda_fp8_matmul_cut(FAKE, K, FAKE + 2 * G, w, K, FAKE + 3 * G, M, N, K, 1, FAKE + 4 * G, N, *cut, None) == want
    assert lib.kda_fp8_matmul_cut(FAKE, K, FAKE + 2 * G, w, K, FAKE + 3 * G, 0, N, K, 1, FAKE + 4 * G, N, *cut, None) == 0
