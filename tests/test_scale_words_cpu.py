"""Scale bytes of a paged cache that are read in aligned words: every word that is read lies in the pool (the library's own
header)."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dropless_moe_expert_router_gb300", "csrc")
SOURCE = """
#include "scale_words.h"
extern "C" int skip(unsigned long long row, int n) { return moe::scale_words(row, n).skip; }
extern "C" int words(unsigned long long row, int n) { return moe::scale_words(row, n).words; }
extern "C" int at_an_end(long long line, long long lines) { return moe::scales_at_an_end(line, lines); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("scale_words")
    src, so = str(d / "t.cpp"), str(d / "t.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.check_call([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, src, "-o", so])
    lib = C.CDLL(so)
    lib.skip.argtypes = lib.words.argtypes = [C.c_ulonglong, C.c_int]
    lib.at_an_end.argtypes = [C.c_longlong, C.c_longlong]
    return lib


@pytest.mark.parametrize("n", range(1, 8))
def test_words_stay_in_the_pool(lib, n):
    align = 4 if n % 4 == 0 else 2 if n % 2 == 0 else 1
    left = 0
    for lines in (1, 2, 3, 5, 6, 7, 8, 24, 100):
        for first in range(4096, 4100, align):
            end = first + lines * n
            for line in range(lines):
                row = first + line * n
                begin = row - lib.skip(row, n)
                last = begin + 4 * lib.words(row, n)
                assert begin % 4 == 0 and begin <= row and row + n <= last and last - begin <= 4 * ((n + 6) // 4)
                inside = first <= begin and last <= end
                left += not inside
                assert inside or lib.at_an_end(line, lines)
    assert (left > 0) == (n != 4)                             # (the rule is needed, but for whole words)


def test_few_rows_are_read_by_their_bytes(lib):
    assert sum(lib.at_an_end(i, 1000) for i in range(1000)) == 6
    assert not lib.at_an_end(1 << 33, 1 << 34) and lib.at_an_end((1 << 34) - 1, 1 << 34)
