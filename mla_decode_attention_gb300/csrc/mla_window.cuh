// Windowed attention: which keys query tokens see and how the work is cut.
// Pure integer arithmetic, compiled for host and device.
//
// A token at position p of its request sees the keys t <= p with t > p - window
// or t < sinks.  A kernel's block of query rows holds the heads of `group`
// consecutive tokens of a request (an item): with few heads several tokens fill
// a block, and they see nearly the same keys.  The pages that hold a key that
// any of them sees are two runs, the first tokens' and the window's (one run
// when they meet); written one after the other they form the item's page list,
// and a 128-key tile is two consecutive entries of that list.  Pages between the
// runs are never touched, and a few first tokens share their tile with the
// window's first page.  Keys of a tile that a token does not see are masked by
// position.
//
// What a call costs beyond its bytes and products is this: a part begins cold
// (code, query rows and first keys: 64 tokens of 128 heads over 128 keys take 18
// us, their bytes 4), and every piece has a cost of its own (its query rows in,
// its output rows out).  So pieces are few and large, and nothing runs before
// the kernel that walks them.
//
// No schedule is built on the device: an item has at most `tiles` tiles, so the
// cost line of all items is known without their lengths.  Each item takes
// fixed + tiles cost units on it, a part walks the units [part * per, (part + 1)
// * per), and an item with fewer tiles scales its range.  With per a multiple of
// an item's cost nothing is cut; otherwise an item on a boundary is cut into
// pieces that the combine merges.  The items are dealt to `lanes` cost lines in
// turn, so that neighbouring items, which share keys, are walked at the same
// time by different parts and find each other's keys in L2.
#pragma once

#include <cstdint>

#include "mla_schedule.cuh"

namespace mla {

constexpr int kWindowPage = 64;
constexpr int32_t kWindowMaxLen = 1 << 30;  // longer lengths are taken as this

// Of the tokens j0 .. j0 + group - 1: the least and the largest end among those
// that are no padding (both 0 when there is none); token j0 + j has end first + j
// when j < count and that is positive, else it is padding.
struct WindowEnds {
  int32_t least, most, first, count;
};
// Of a request of length L, n of whose s slots hold new tokens.
MLA_HD WindowEnds item_ends(int32_t L, int32_t n, int s, int j0, int group) {
  n = n < 0 ? 0 : (n > s ? s : n);
  L = L > kWindowMaxLen ? kWindowMaxLen : (L < 0 ? 0 : L);
  const int32_t last = (j0 + group < n ? j0 + group : n) - 1;  // the last token that is not past the new ones
  WindowEnds e;
  e.first = L - n + j0 + 1;
  e.count = last - j0 + 1;
  e.most = L - n + last + 1;
  e.least = e.first > 1 ? e.first : 1;
  if (e.count <= 0 || L <= 0 || e.most <= 0) e.least = e.most = e.count = 0;
  return e;
}
MLA_HD WindowEnds window_ends(const int32_t* seqlens, const int32_t* new_lens, int s, int b, int j0, int group) {
  return item_ends(seqlens[b], new_lens ? new_lens[b] : s, s, j0, group);
}

// End (one past the position) of token j of an item, 0 for padding.
MLA_HD int32_t item_end(int32_t first, int32_t count, int32_t j) { return j < count && first + j > 0 ? first + j : 0; }
// Of token j of request b, as the item of all its tokens has it.
MLA_HD int32_t window_end(const int32_t* seqlens, const int32_t* new_lens, int s, int b, int j) {
  const WindowEnds e = window_ends(seqlens, new_lens, s, b, 0, s);
  return item_end(e.first, e.count, j);
}

// Length of request b and how many of its s slots hold new tokens, read past L1;
// with `read` false made up, and nothing is read.
struct RequestLengths {
  int32_t L, n;
};
constexpr int32_t kDryLength = 1 << 20;
MLA_HD RequestLengths request_lengths(const int32_t* seqlens, const int32_t* new_lens, int s, int b, bool read) {
  if (!read) return {kDryLength, s};
#ifdef __CUDA_ARCH__
  return {__ldcg(seqlens + b), new_lens ? __ldcg(new_lens + b) : s};
#else
  return {seqlens[b], new_lens ? new_lens[b] : s};
#endif
}

MLA_HD int32_t window_lo(int32_t end, int32_t window) { return end > window ? end - window : 0; }
MLA_HD uint32_t low_bits(int32_t n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }
// Whether a token with this end sees key t; bit i of the mask: key x + i.
MLA_HD bool window_sees(int32_t end, int32_t window, int32_t sinks, int32_t t) {
  return t < end && (t < sinks || t >= window_lo(end, window));
}
MLA_HD uint32_t window_mask32(int32_t end, int32_t window, int32_t sinks, int32_t x) {
  return low_bits(end - x) & (low_bits(sinks - x) | ~low_bits(window_lo(end, window) - x));
}

// The page list of an item.
struct WindowSpan {
  int32_t head_pages;  // entries of the first tokens' run
  int32_t skip;        // pages between the two runs
  int32_t tiles;
  // tiles that may hold a key that one of the tokens does not see: the one with
  // the last of the first tokens, those with the tokens' first window keys, and
  // from the one with the first token's last key on
  int32_t edge_head, edge_lo, edge_hi, edge_end;

  // logical page of entry e of the list
  MLA_HD int32_t page(int32_t e) const { return e < head_pages ? e : e + skip; }
  MLA_HD bool edge(int32_t t) const { return t == edge_head || (t >= edge_lo && t <= edge_hi) || t >= edge_end; }
};

MLA_HD WindowSpan window_span(WindowEnds e, int32_t window, int32_t sinks) {
  WindowSpan w;
  const int32_t lo = window_lo(e.least, window), lo_most = window_lo(e.most, window);
  const bool two = sinks > 0 && sinks < lo;  // the runs of keys do not meet
  w.head_pages = two ? (sinks - 1) / kWindowPage + 1 : 0;
  const int32_t first_page = (sinks > 0 && !two) ? 0 : lo / kWindowPage;
  w.skip = first_page > w.head_pages ? first_page - w.head_pages : 0;
  const int32_t pages = e.most > 0 ? (e.most - 1) / kWindowPage + 1 - w.skip : 0;
  w.tiles = (pages + 1) / 2;
  w.edge_head = sinks > 0 && sinks < lo_most ? (sinks - 1) / kWindowPage / 2 : -1;
  w.edge_lo = lo_most > 0 ? (lo / kWindowPage - w.skip) / 2 : 0;
  w.edge_hi = lo_most > 0 ? (lo_most / kWindowPage - w.skip) / 2 : -1;
  const int32_t from = (e.least / kWindowPage - w.skip) / 2;
  w.edge_end = from < w.tiles - 1 ? from : w.tiles - 1;
  return w;
}

// The most tiles that an item of `group` tokens can have.
MLA_HD int32_t window_max_tiles(int32_t window, int32_t sinks, int32_t group) {
  const int64_t w = (window < kWindowMaxLen ? window : kWindowMaxLen) + static_cast<int64_t>(group) - 1;
  const int64_t k = sinks < kWindowMaxLen ? sinks : kWindowMaxLen;
  const int64_t pages = (w + kWindowPage - 2) / kWindowPage + 1 + (k + kWindowPage - 1) / kWindowPage;
  return static_cast<int32_t>((pages + 1) / 2);
}

// How a call's items are laid on the cost lines and cut.
struct WindowPlan {
  int32_t group;   // tokens per item
  int32_t chunks;  // items per request
  int32_t items;
  int32_t parts;
  int32_t tiles;   // of an item on the cost line
  int32_t fixed;   // cost of an item besides its tiles
  int32_t lanes;   // cost lines: item i is number i / lanes of line i % lanes; part p is number p / lanes of line p % lanes
  int64_t per;     // cost units per part
  bool whole;      // per is a multiple of an item's cost: nothing is cut
};

// Piece of item number m of a line that the line's part number pl walks, out of
// n_tiles tiles: [t0, t1), empty when t0 >= t1.
struct WindowPiece {
  int32_t t0, t1;
  bool owner;  // the part with the item's first unit: it writes items without a key
  bool cut;    // other parts walk tiles of the item too
};
MLA_HD int32_t window_scaled(int64_t unit, int32_t n_tiles, int32_t tiles) {
  return tiles == n_tiles ? static_cast<int32_t>(unit) : static_cast<int32_t>(floordiv(unit * n_tiles, tiles));
}
MLA_HD WindowPiece window_piece(const WindowPlan& w, int64_t m, int64_t pl, int32_t n_tiles) {
  if (w.whole) return {0, n_tiles, true, false};
  const int64_t at = m * (w.tiles + w.fixed) + w.fixed;  // the unit of its first tile
  const int64_t x0 = pl * w.per - at, x1 = x0 + w.per;
  const int64_t b = x0 > 0 ? x0 : 0, e = x1 < w.tiles ? x1 : w.tiles;
  WindowPiece p;
  p.owner = x0 <= 0 && x1 > 0;
  p.cut = b > 0 || e < w.tiles;
  p.t0 = p.t1 = 0;
  if (b < e) {
    p.t0 = window_scaled(b, n_tiles, w.tiles);
    p.t1 = window_scaled(e, n_tiles, w.tiles);
  }
  return p;
}
// First item number that part number pl walks (0 for whole items: every line has
// one part), and the line's parts that walk tiles of item number m.
MLA_HD int64_t window_first_item(const WindowPlan& w, int64_t pl) {
  return w.whole ? 0 : floordiv(pl * w.per, w.tiles + w.fixed);
}
MLA_HD int64_t window_first_part(const WindowPlan& w, int64_t m) {
  return floordiv(m * (w.tiles + w.fixed) + w.fixed, w.per);
}
MLA_HD int64_t window_last_part(const WindowPlan& w, int64_t m) {
  return floordiv((m + 1) * (w.tiles + w.fixed) - 1, w.per);
}
// Workspace block of a cut item's piece: a part walks at most two such pieces,
// of the item in whose units it begins and of another at its end.
MLA_HD int32_t window_row(const WindowPlan& w, int64_t m, int64_t pl, int32_t lane) {
  return static_cast<int32_t>(2 * (pl * w.lanes + lane) + (window_first_item(w, pl) == m ? 0 : 1));
}

// The two-SM kernel requests every piece's query rows as four boxes, in the order
// 0, 2, 1, 3: loads of box i among the first n boxes requested.
MLA_HD uint32_t q_box_loads(uint32_t n, int i) {
  const uint32_t place = i == 1 ? 2u : (i == 2 ? 1u : static_cast<uint32_t>(i));
  return (n + 3u - place) / 4u;
}

// fixed: what a piece costs besides its tiles (query load, epilogue), and
// merge: what writing partial rows and merging them costs a call, in tiles.
inline WindowPlan window_plan(int batch, int s_q, int group, int window, int sinks, int parts, bool ragged, int fixed,
                              int merge) {
  WindowPlan w;
  w.group = group;
  w.chunks = (s_q + group - 1) / group;
  w.items = batch * w.chunks;
  w.tiles = window_max_tiles(window, sinks, group);
  w.fixed = fixed;
  const int64_t cost = static_cast<int64_t>(w.tiles) + fixed;
  // whole items, dealt round
  const int lines = w.items < parts ? w.items : parts;
  const int64_t whole = (w.items + lines - 1) / lines * cost;
  w.parts = w.lanes = lines;
  w.per = whole;
  w.whole = true;
  // cut into equal parts; with new_lens many items may be padding, and only
  // dealing whole items round spreads them evenly
  if (ragged && w.items >= parts) return w;
  int64_t best = 0;
  int best_lanes = 1;
  for (int lanes = 1; lanes <= 16 && lanes <= w.chunks && lanes <= parts; ++lanes) {
    const int64_t line = (w.items + lanes - 1) / lanes * cost;
    const int64_t n = parts / lanes;
    const int64_t per = (line + n - 1) / n;
    if (lanes == 1) best = per;
    if (per * 20 <= best * 21) best_lanes = lanes;  // shared keys are worth 5 %
  }
  const int64_t n = parts / best_lanes;
  const int64_t per = ((w.items + best_lanes - 1) / best_lanes * cost + n - 1) / n;
  // few items: each into the same number of pieces, a part each
  const int pieces = parts / w.items < w.tiles ? parts / w.items : w.tiles;
  const int64_t each = pieces > 1 ? (static_cast<int64_t>(w.tiles) + pieces - 1) / pieces : 0;
  if (each > 0 && each <= per && each + fixed + merge < whole) {
    w.parts = parts;
    w.lanes = 1;
    w.per = each;
    w.tiles = static_cast<int32_t>(each * pieces);
    w.fixed = 0;
    w.whole = false;
  } else if (per + fixed + merge < whole) {
    w.parts = parts;
    w.lanes = best_lanes;
    w.per = per;
    w.whole = false;
  }
  return w;
}

}  // namespace mla
