"""Index arithmetic of the attention kernels over the paged cache, compiled for the
host and checked over its whole range: sequences of up to 2^31 - 1 tokens in pages of
16 to 4096."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_recurrence_chunk_gb300",
                    "csrc", "kv4")

SOURCE = r"""
#include "index.cuh"
using namespace kda::kv4;
extern "C" {
// The first unit of 0 .. n - 1 whose page is not unit / upp, or -1.  (The page does not
// fall as the unit grows, so both ends of every page show it.)
int64_t first_wrong_page(uint32_t upp, int64_t n) {
  const uint64_t inv = page_inverse(upp);
  for (int64_t u = 0; u < n; u += upp) {
    const int64_t last = u + upp - 1 < n ? u + upp - 1 : n - 1;
    if (page_of_unit((uint32_t)u, inv) != u / upp) return u;
    if (page_of_unit((uint32_t)last, inv) != u / upp) return last;
  }
  return -1;
}
int64_t token(int64_t i, int32_t tokens, int32_t at) { return token_of_tile(i, tokens, at); }
int32_t blocks(int32_t qn, int32_t G, int32_t R) { return row_blocks(qn, G, R); }
int32_t units(int32_t L, int32_t i, int32_t most) { return units_of_tile(L, i, most); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4_index")
    (d / "index.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", CSRC, str(d / "index.cpp"), "-o", str(d / "index.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "index.so"))
    lib.first_wrong_page.argtypes, lib.first_wrong_page.restype = [ctypes.c_uint32, ctypes.c_int64], ctypes.c_int64
    lib.token.argtypes, lib.token.restype = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32], ctypes.c_int64
    lib.units.argtypes, lib.units.restype = [ctypes.c_int32] * 3, ctypes.c_int32
    lib.blocks.argtypes, lib.blocks.restype = [ctypes.c_int32] * 3, ctypes.c_int32
    return lib


UNITS = 1 << 27   # of 2^31 - 1 tokens


@pytest.mark.parametrize("upp", [1, 2, 3, 4, 5, 7, 8, 16, 31, 64, 100, 128, 255, 256])
def test_page_of_a_unit(lib, upp):
    assert lib.first_wrong_page(upp, UNITS) == -1


def test_page_of_a_unit_every_page_size(lib):
    """The other page sizes at their last pages, where an inverse that is cut off too early shows first."""
    for upp in range(1, 257):
        assert lib.first_wrong_page(upp, 1 << 20) == -1, upp


MOST = (1 << 31) - 1


@pytest.mark.parametrize("L", [1, 127, 128, 129, 1 << 28, MOST - 512, MOST - 127, MOST])
def test_tokens_loaded_ahead(lib, L):
    """The tiles of 128 tokens up to two behind the last: every token keeps its place, below L or not."""
    last = (L - 1) // 128
    for i in range(max(last - 3, 0), last + 3):
        for at in (0, 1, 64, 127):
            assert lib.token(i, 128, at) == 128 * i + at


@pytest.mark.parametrize("L", [0, 1, 16, 17, 63, 64, 65, 1 << 28, MOST - 65, MOST - 16, MOST - 15, MOST])
def test_units_of_a_tile(lib, L):
    tiles = max(-(-L // 64), 1)
    for i in range(max(tiles - 3, 0), tiles):
        assert lib.units(L, i, 4) == min(4, -(-L // 16) - 4 * i)
    assert L == 0 or 1 <= lib.units(L, tiles - 1, 4) <= 4


@pytest.mark.parametrize("qn,G", [(0, 1), (0, 128), (1, 1), (8, 1), (3, 12), (2048, 4), (MOST, 1), (MOST - 7, 1), (MOST // 12, 12), (MOST // 128, 128)])
def test_row_blocks(lib, qn, G):
    for R in (8, 16):
        assert lib.blocks(qn, G, R) == -(-qn * G // R)
