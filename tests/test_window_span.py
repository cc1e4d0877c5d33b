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
using namespace mla;
static WindowEnds ends(int least, int most) { WindowEnds e; e.least = least; e.most = most; return e; }
extern "C" {
int tiles(int least, int most, int window, int sinks) { return window_span(ends(least, most), window, sinks).tiles; }
int max_tiles(int window, int sinks, int group) { return window_max_tiles(window, sinks, group); }
// logical pages of tile t and whether it may hold a key that a token does not see
int tile(int least, int most, int window, int sinks, int t, int* pages) {
  const WindowSpan w = window_span(ends(least, most), window, sinks);
  for (int h = 0; h < 2; ++h) pages[h] = w.page(2 * t + h);
  return w.edge(t);
}
// the 128 keys of two pages that a token sees; -1: the two forms disagree
int seen(int end, int window, int sinks, const int* pages, unsigned* bits) {
  for (int k = 0; k < 4; ++k) bits[k] = window_mask32(end, window, sinks, 64 * pages[k >> 1] + 32 * (k & 1));
  for (int i = 0; i < 128; ++i)
    if (window_sees(end, window, sinks, 64 * pages[i >> 6] + (i & 63)) != ((bits[i >> 5] >> (i & 31)) & 1)) return -1;
  return 0;
}
int end_of(const int* lens, const int* fresh, int s, int b, int j) { return window_end(lens, fresh, s, b, j); }
void ends_of(const int* lens, const int* fresh, int s, int b, int j0, int group, int* out) {
  const WindowEnds e = window_ends(lens, fresh, s, b, j0, group);
  out[0] = e.least; out[1] = e.most;
}
static WindowPlan plan;
void make(int batch, int s, int group, int window, int sinks, int parts, int ragged, int fixed, int cut, long long* out) {
  plan = window_plan(batch, s, group, window, sinks, parts, ragged, fixed, cut);
  out[0] = plan.items; out[1] = plan.tiles; out[2] = plan.lanes; out[3] = plan.per; out[4] = plan.whole; out[5] = plan.parts;
}
// the walk of a part as the kernels do it: (item, t0, t1, cut, workspace block, owner) each
int walk(int part, const int* item_tiles, int* out) {
  const int lane = part % plan.lanes, pl = part / plan.lanes;
  int n = 0;
  for (long long m = window_first_item(plan, pl);; ++m) {
    const long long item = lane + plan.lanes * m;
    if (item >= plan.items || m * (plan.tiles + plan.fixed) >= (pl + 1) * plan.per) return n;
    const WindowPiece p = window_piece(plan, m, pl, item_tiles[item]);
    int* o = out + 6 * n++;
    o[0] = item; o[1] = p.t0; o[2] = p.t1; o[3] = p.cut; o[4] = p.cut ? window_row(plan, m, pl, lane) : -1; o[5] = p.owner;
  }
}
// the merge's view of a part: the cut item that begins in it, its pieces' blocks
int merge(int part, const int* item_tiles, int* blocks) {
  const int lane = part % plan.lanes, pl = part / plan.lanes;
  const long long m = floordiv((pl + 1) * plan.per - 1, plan.tiles + plan.fixed), item = lane + plan.lanes * m;
  if (item >= plan.items || window_first_part(plan, m) != pl || window_last_part(plan, m) == pl) return -1;
  for (long long i = pl; i <= window_last_part(plan, m); ++i) {
    const WindowPiece p = window_piece(plan, m, i, item_tiles[item]);
    blocks[i - pl] = p.t0 < p.t1 ? window_row(plan, m, i, lane) : -1;
  }
  blocks[window_last_part(plan, m) - pl + 1] = -2;
  return item;
}
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


def check_item(lib, ends, window, sinks):
    """The tile list of an item whose tokens have these ends shows every token
    exactly its keys, once; every tile shows some token one, and a tile that is
    not marked as an edge shows every token all of its keys."""
    shown = {e: [] for e in ends}
    for t in range(lib.tiles(ends[0], ends[-1], window, sinks)):
        pages = (ctypes.c_int * 2)()
        edge = lib.tile(ends[0], ends[-1], window, sinks, t, pages)
        some = 0
        for e in ends:
            bits = (ctypes.c_uint * 4)()
            assert lib.seen(e, window, sinks, pages, bits) == 0
            here = [64 * pages[i >> 6] + (i & 63) for i in range(128) if (bits[i >> 5] >> (i & 31)) & 1]
            assert edge or len(here) == 128, (ends, window, sinks, t)
            some += len(here)
            shown[e] += here
        assert some, (ends, window, sinks, t)
    for e in ends:
        want = oracle.window_keys(e - 1, window, sinks)
        assert sorted(shown[e]) == want.tolist(), (ends, e, window, sinks)
    return lib.tiles(ends[0], ends[-1], window, sinks)


SIZES = [1, 2, 63, 64, 65, 127, 128, 129, 200, 500]
ENDS = list(range(1, 140)) + [191, 192, 193, 255, 256, 257, 300, 511, 512, 513, 700, 1000, 1001]


@pytest.mark.parametrize("window", SIZES + [2**31 - 1])
def test_tiles_show_exactly_the_visible_keys(spans, window):
    for sinks in [0] + SIZES + [2**31 - 1]:
        assert spans.tiles(0, 0, window, sinks) == 0
        most = max(check_item(spans, [end], window, sinks) for end in ENDS)
        assert most <= spans.max_tiles(window, sinks, 1)


@pytest.mark.parametrize("window", [1, 7, 64, 65, 128, 200, 2**31 - 1])
def test_items_of_several_tokens(spans, window):
    for sinks in [0, 1, 4, 63, 64, 65, 127, 128, 129, 192, 300, 2**31 - 1]:
        for group in (2, 3, 8):
            for end in [1, 2, 60, 61, 62, 63, 64, 65, 120, 121, 126, 127, 128, 129, 190, 250, 256, 257, 320, 450, 511, 513]:
                n = check_item(spans, list(range(end, end + group)), window, sinks)
                assert n <= spans.max_tiles(window, sinks, group)


def test_pages_between_the_runs_are_left_out(spans):
    # 4 first tokens (1 page) and a window of 128 at position 100000 (3 pages): two tiles
    assert spans.tiles(100001, 100001, 128, 4) == 2
    assert spans.tiles(100001, 100001, 2**31 - 1, 0) == (100001 + 127) // 128


PLANS = [(1, 1, 1, 128, 4), (3, 1, 1, 8192, 128), (64, 1, 1, 4096, 0), (128, 2, 1, 4096, 64), (77, 1, 1, 1000, 0), (2, 5, 2, 300, 0),
         (1, 1000, 8, 512, 0), (7, 3, 1, 2**31 - 1, 0), (256, 1, 1, 128, 4), (9, 16, 4, 70, 2)]


@pytest.mark.parametrize("shape", PLANS)
@pytest.mark.parametrize("parts", [1, 2, 5, 76, 152])
def test_parts_cover_every_tile_once(spans, shape, parts):
    """Whatever the items' own lengths: every tile of every item is in one piece,
    cut pieces have blocks of the workspace of their own, the merge finds them,
    and one part owns each item."""
    batch, s, group, window, sinks = shape
    rng = np.random.default_rng(parts)
    for ragged in (0, 1):
        info = (ctypes.c_longlong * 6)()
        spans.make(batch, s, group, window, sinks, parts, ragged, 5, 8, info)
        items, tiles, lanes, per, whole, used = list(info)
        assert 1 <= used <= parts and lanes <= used
        assert items == batch * -(-s // group) and tiles >= spans.max_tiles(window, sinks, group)
        for kind in range(3):
            most = min(tiles, 300)
            n_tiles = np.full(items, tiles if tiles < 300 else 7) if kind == 0 else rng.integers(0, most + 1, items)
            if kind == 2:
                n_tiles = np.minimum(n_tiles, 2)
            arr = (ctypes.c_int * items)(*n_tiles.tolist())
            covered = {i: [] for i in range(items)}
            blocks, owners = {}, {}
            for part in range(used):
                out = (ctypes.c_int * (6 * (2 * items + 8)))()
                for k in range(spans.walk(part, arr, out)):
                    item, t0, t1, cut, block, owner = out[6 * k:6 * k + 6]
                    owners[item] = owners.get(item, 0) + owner
                    if t0 < t1:
                        covered[item] += range(t0, t1)
                        assert not (whole and cut)
                        if cut:
                            assert 0 <= block < 2 * parts and block not in blocks
                            blocks[block] = item
                        else:
                            assert (t0, t1) == (0, n_tiles[item])
            assert all(sorted(covered[i]) == list(range(n_tiles[i])) for i in range(items))
            assert owners == {i: 1 for i in range(items)}
            merged = {}
            for part in range(used):
                out = (ctypes.c_int * (parts + 2))()
                item = spans.merge(part, arr, out)
                if item >= 0:
                    assert item not in merged
                    row = list(out)
                    merged[item] = [x for x in row[:row.index(-2)] if x >= 0]
            for item in set(blocks.values()):
                assert sorted(merged[item]) == sorted(k for k, v in blocks.items() if v == item)
            assert sum(map(len, merged.values())) == len(blocks)


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
                    for group in (1, 2, 3, 4):
                        out = (ctypes.c_int * 2)()
                        spans.ends_of(arr, new, s, b, j, group, out)
                        real = [e for e in want[b, j:j + group] if e > 0]
                        assert list(out) == ([min(real), max(real)] if real else [0, 0]), (b, j, group, fresh)
    # lengths past 2^30 count as 2^30
    assert spans.end_of((ctypes.c_int * 1)(2**31 - 1), None, 1, 0, 0) == 2**30
