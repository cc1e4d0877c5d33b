"""Lengths as the windowed decode's planning warp takes them, on the CPU
(csrc/mla_window.cuh compiled as plain C++): before its wait for the kernel
ahead in the stream it must not look at them at all."""
import ctypes
import os
import shutil
import subprocess

import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "mla_window.cuh"
using namespace mla;
extern "C" void lengths(const int* lens, const int* fresh, int s, int b, int read, int* out) {
  const RequestLengths r = request_lengths(lens, fresh, s, b, read != 0);
  out[0] = r.L; out[1] = r.n;
}
extern "C" int end(int first, int count, int j) { return item_end(first, count, j); }
extern "C" void ends(int L, int n, int s, int j0, int group, int* out) {
  const WindowEnds e = item_ends(L, n, s, j0, group);
  out[0] = e.least; out[1] = e.most; out[2] = e.first; out[3] = e.count;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("lengths")
    (d / "lengths.cpp").write_text(SOURCE)
    out = str(d / "lengths.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "mla_decode_attention_gb300", "csrc"),
                    str(d / "lengths.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def test_nothing_is_read_before_the_wait(lib):
    """Addresses that no read would survive."""
    out = (ctypes.c_int * 2)()
    for s in (1, 5):
        lib.lengths(ctypes.c_void_p(8), ctypes.c_void_p(8), s, 3, 0, out)
        assert out[0] >= s and out[1] == s


def test_what_is_read_after_it(lib):
    lens, fresh, out = (ctypes.c_int * 4)(7, 0, -3, 2**31 - 1), (ctypes.c_int * 4)(1, 9, -2, 3), (ctypes.c_int * 2)()
    for b in range(4):
        lib.lengths(lens, fresh, 5, b, 1, out)
        assert list(out) == [lens[b], fresh[b]]
        lib.lengths(lens, None, 5, b, 1, out)
        assert list(out) == [lens[b], 5]


def test_ends_of_items(lib):
    out = (ctypes.c_int * 4)()
    for L in (-1, 0, 1, 2, 3, 5, 64, 200):
        for s in (1, 2, 7):
            for n in (-1, 0, 1, 2, s, s + 3):
                pos = oracle.token_positions([L], [n], s)[0]
                for group in (1, 2, 4):
                    for j0 in range(0, s, group):
                        lib.ends(L, n, s, j0, group, out)
                        real = [int(p) + 1 for p in pos[j0:j0 + group] if p >= 0]
                        assert list(out)[:2] == ([min(real), max(real)] if real else [0, 0]), (L, s, n, j0, group)
                        # the query rows of the item: of each token, and of rows past the last one
                        for j in range(group):
                            p = int(pos[j0 + j]) if j0 + j < s else -1
                            assert lib.end(out[2], out[3], j) == p + 1, (L, s, n, j0, group, j)
