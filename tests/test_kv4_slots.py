"""The page of a position, for every page size and up to the last position that a table may name (no GPU)."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "streaming_persistent_sm_b200", "csrc")

# Every first and last position of a page, against a division in 64 bits; the first wrong one, or -1.  The quotient
# does not fall as positions rise (nor does a product shifted down), so what holds at both ends holds between them.
SOURCE = r"""
#include "kv4_slot.h"
extern "C" long long first_wrong(int page) {
  const uint64_t magic = wpk::kv4_page_magic(page);
  const long long end = 2147483647ll;
  for (long long slot = 0; slot * page <= end; ++slot) {
    const long long first = slot * page, last = first + page - 1 < end ? first + page - 1 : end;
    if (wpk::kv4_slot_of((int)first, magic) != slot) return first;
    if (wpk::kv4_slot_of((int)last, magic) != slot) return last;
  }
  return -1;
}
"""


@pytest.fixture(scope="module")
def first_wrong(tmp_path_factory):
    d = tmp_path_factory.mktemp("slots")
    (d / "slots.cpp").write_text(SOURCE)
    so = str(d / "slots.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "slots.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).first_wrong
    f.restype = ctypes.c_longlong
    return f


@pytest.mark.parametrize("page", range(16, 257, 16))
def test_every_position_finds_its_page(first_wrong, page):
    assert first_wrong(page) == -1
