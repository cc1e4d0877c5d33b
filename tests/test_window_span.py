"""The windowed decode's tile lists on the CPU: csrc/mla_window.cuh compiled as
plain C++ and compared with the definition (key t of the token at position p is
seen when t <= p and (t > p - window or t < sinks)), written out key by key."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "mla_window.cuh"
extern "C" {
int tiles(int end, int window, int sinks) { return mla::window_span(end, window, sinks).tiles; }
int max_tiles(int window, int sinks) { return mla::window_max_tiles(window, sinks); }
// logical pages and the 128 seen bits of tile t
void tile(int end, int window, int sinks, int t, int* pages, unsigned* bits, int* edge) {
  const mla::WindowSpan w = mla::window_span(end, window, sinks);
  for (int h = 0; h < 2; ++h) {
    pages[h] = w.page(2 * t + h);
    for (int k = 0; k < 2; ++k) bits[2 * h + k] = w.mask32(64 * pages[h] + 32 * k);
  }
  *edge = w.edge(t);
  for (int i = 0; i < 128; ++i)  // the two forms of the mask agree
    if (w.sees(64 * pages[i >> 6] + (i & 63)) != ((bits[i >> 5] >> (i & 31)) & 1)) *edge = -1;
}
void piece(int tiles, int pieces, int split, int* t0, int* t1) { mla::window_piece(tiles, pieces, split, t0, t1); }
int end_of(const int* lens, const int* fresh, int s, int b, int j) { return mla::window_end(lens, fresh, s, b, j); }
}
"""


@pytest.fixture(scope="module")
def spans(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("span")
    (d / "span.cpp").write_text(SOURCE)
    lib = str(d / "span.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "mla_decode_attention_gb300", "csrc"), str(d / "span.cpp"), "-o", lib], check=True)
    return ctypes.CDLL(lib)


def seen_by_tiles(lib, end, window, sinks):
    """Positions that the tile list shows, tile by tile; every tile shows one."""
    found = []
    for t in range(lib.tiles(end, window, sinks)):
        pages, bits, edge = (ctypes.c_int * 2)(), (ctypes.c_uint * 4)(), ctypes.c_int()
        lib.tile(end, window, sinks, t, pages, bits, ctypes.byref(edge))
        here = [64 * pages[i >> 6] + (i & 63) for i in range(128) if (bits[i >> 5] >> (i & 31)) & 1]
        assert here, "a tile without a visible key"
        assert edge.value >= 0 and (edge.value or len(here) == 128)
        found += here
    return found


SIZES = [1, 2, 63, 64, 65, 127, 128, 129, 200, 500]


@pytest.mark.parametrize("window", SIZES + [2**31 - 1])
def test_tiles_show_exactly_the_visible_keys(spans, window):
    for sinks in [0] + SIZES + [2**31 - 1]:
        most = 0
        for end in list(range(0, 140)) + [191, 192, 193, 255, 256, 257, 300, 511, 512, 513, 700, 1000, 1001]:
            want = oracle.window_keys(end - 1, window, sinks)
            got = seen_by_tiles(spans, end, window, sinks)
            assert sorted(got) == want.tolist(), (end, window, sinks)
            assert len(set(got)) == len(got)
            most = max(most, spans.tiles(end, window, sinks))
        assert most <= spans.max_tiles(window, sinks)


def test_pages_between_the_runs_are_left_out(spans):
    # 4 first tokens (1 page) and a window of 128 at position 100000 (3 pages): two tiles
    assert spans.tiles(100001, 128, 4) == 2
    assert spans.tiles(100001, 2**31 - 1, 0) == (100001 + 127) // 128


def test_pieces_cover_the_tiles(spans):
    for tiles in range(1, 40):
        for pieces in range(1, tiles + 1):
            at = 0
            for k in range(pieces):
                t0, t1 = ctypes.c_int(), ctypes.c_int()
                spans.piece(tiles, pieces, k, ctypes.byref(t0), ctypes.byref(t1))
                assert t0.value == at and t1.value > at
                at = t1.value
            assert at == tiles


def test_token_ends(spans):
    lens = [0, 1, 3, 10, -4, 2**31 - 1]
    for fresh in (None, [4, 4, 2, 0, 4, 1], [9, -1, 5, 3, 0, 4]):
        for s in (1, 4):
            want = oracle.token_positions(lens, fresh, s) + 1
            arr = (ctypes.c_int * 6)(*lens)
            new = None if fresh is None else (ctypes.c_int * 6)(*fresh)
            for b in range(5):
                for j in range(s):
                    assert spans.end_of(arr, new, s, b, j) == want[b, j], (b, j, fresh)
    # lengths past 2^30 count as 2^30
    assert spans.end_of((ctypes.c_int * 1)(2**31 - 1), None, 1, 0, 0) == 2**30
