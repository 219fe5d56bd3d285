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
    return lib


UNITS = 1 << 27   # of 2^31 - 1 tokens


@pytest.mark.parametrize("upp", [1, 2, 3, 4, 5, 7, 8, 16, 31, 64, 100, 128, 255, 256])
def test_page_of_a_unit(lib, upp):
    assert lib.first_wrong_page(upp, UNITS) == -1


def test_page_of_a_unit_every_page_size(lib):
    """The other page sizes at their last pages, where an inverse that is cut off too early shows first."""
    for upp in range(1, 257):
        assert lib.first_wrong_page(upp, 1 << 20) == -1, upp
