// Windowed attention: which keys a query token sees and how its work is cut.
// Pure integer arithmetic, compiled for host and device.
//
// A token at position p of its request sees the keys t <= p with t > p - window
// or t < sinks.  The pages that hold any of them are two runs, the first
// tokens' and the window's (one run when they meet); written one after the
// other they form the token's page list, and a 128-key tile is two consecutive
// entries of that list.  So a tile always holds a visible key, pages between
// the runs are never touched, and a few first tokens share their tile with the
// window's first page.  Keys of a tile that the token does not see are masked
// by position.
//
// No schedule is needed: a token has at most window / 128 + 2 tiles (and the
// first tokens'), so every token's list is cut into the same number of pieces,
// chosen on the host, and part i walks the pieces i, i + parts, ...
// Neighbouring tokens of a request are walked at the same time and find each
// other's keys in L2.
#pragma once

#include <cstdint>

#include "mla_schedule.cuh"

namespace mla {

constexpr int kWindowPage = 64;
constexpr int32_t kWindowMaxLen = 1 << 30;  // longer lengths are taken as this

// Token j of request b: one past its position, or 0 for padding (slots past
// new_lens[b], positions before the first).
MLA_HD int32_t window_end(const int32_t* seqlens, const int32_t* new_lens, int s, int b, int j) {
  int32_t n = new_lens ? new_lens[b] : s;
  n = n < 0 ? 0 : (n > s ? s : n);
  int32_t L = seqlens[b];
  L = L > kWindowMaxLen ? kWindowMaxLen : L;
  const int32_t end = L - n + j + 1;
  return (j >= n || L <= 0 || end < 0) ? 0 : end;
}

struct WindowSpan {
  int32_t end, lo, first;  // key t is seen when t < end and (t < first or t >= lo)
  int32_t head_pages;      // list entries of the first tokens' run
  int32_t skip;            // pages between the two runs
  int32_t tiles;

  // logical page of entry e of the list
  MLA_HD int32_t page(int32_t e) const { return e < head_pages ? e : e + skip; }
  MLA_HD bool sees(int32_t t) const { return t < end && (t < first || t >= lo); }
  // bit i: key x + i is seen
  MLA_HD uint32_t mask32(int32_t x) const { return low_bits(end - x) & (low_bits(first - x) | ~low_bits(lo - x)); }
  // Whether tile t may hold a key that is not seen: the tiles with the last of
  // the first tokens, with the window's first key and with the last key.
  MLA_HD bool edge(int32_t t) const {
    return t == tiles - 1 || (lo > 0 && t == (lo / kWindowPage - skip) / 2) ||
           (first > 0 && t == (first - 1) / kWindowPage / 2);
  }
  MLA_HD static uint32_t low_bits(int32_t n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }
};

MLA_HD WindowSpan window_span(int32_t end, int32_t window, int32_t sinks) {
  WindowSpan w;
  w.end = end;
  w.lo = end > window ? end - window : 0;
  w.first = sinks < w.lo ? sinks : 0;
  if (sinks >= w.lo) w.lo = 0;  // the two runs of keys meet: everything is seen
  w.head_pages = w.first > 0 ? (w.first - 1) / kWindowPage + 1 : 0;
  const int32_t first_page = w.lo / kWindowPage;
  w.skip = first_page > w.head_pages ? first_page - w.head_pages : 0;
  const int32_t pages = end > 0 ? (end - 1) / kWindowPage + 1 - w.skip : 0;
  w.tiles = (pages + 1) / 2;
  return w;
}

// The most tiles that any token can have.
MLA_HD int32_t window_max_tiles(int32_t window, int32_t sinks) {
  const int64_t w = window < kWindowMaxLen ? window : kWindowMaxLen, k = sinks < kWindowMaxLen ? sinks : kWindowMaxLen;
  const int64_t pages = (w + kWindowPage - 2) / kWindowPage + 1 + (k + kWindowPage - 1) / kWindowPage;
  return static_cast<int32_t>((pages + 1) / 2);
}

// Piece `split` of n_split of a token's tiles: [t0, t1); a token with fewer
// tiles than n_split has one piece a tile.
MLA_HD int32_t window_pieces(int32_t tiles, int32_t n_split) { return tiles < n_split ? tiles : n_split; }
MLA_HD void window_piece(int32_t tiles, int32_t pieces, int32_t split, int* t0, int* t1) {
  *t0 = static_cast<int>(static_cast<int64_t>(split) * tiles / pieces);
  *t1 = static_cast<int>(static_cast<int64_t>(split + 1) * tiles / pieces);
}

}  // namespace mla
