// Attention of packed sequences with keys and values per head (sm_103a): what a
// prompt's tokens run before absorption pays.
//
//   s = scale * (q[0:128] . k + q[128:192] . k_rope),  out = sum softmax(s) v,
//   lse = ln sum e^s
//
// over the keys t of the query's own sequence, causal to the sequences' ends or all
// of them.  Absorbed, a pair of query head and key costs 2 * (576 + 512) flops; here 2
// * (192 + 128).
//
// A block works on two tiles of 128 query rows and walks the sequence's keys in tiles
// of 128.  A row is one (token, query head of the key head's group) pair, token by
// token, so the heads that share keys fill a tile together.  TMEM holds S0, S1 (the
// tiles' scores, overwritten by their probabilities in bf16) and O0, O1: all 512
// columns.  While the softmax warps of one tile turn S into P, the tensor cores work on the
// other tile's products.  One pass over S with a reference that hardly ever moves: the
// probabilities' fp32 sum divides O (dividing by the sum of the rounded ones instead, as the
// decode kernels do, would take the rounding of a weight that dominates its row, 2^-9 at most, out of
// the output, and costs 5 to 8 % here: softmax is on the products' way).
//
// The query rows stay in shared memory (96 KB, 64 KB without position columns); keys and
// values come through one ring of 16 KB chunks [128 tokens x 64 columns] in the order
// K(0), V(0), K(1), V(1), ... (1.6 key tiles, or 2.5), the position columns that the heads share as
// the third chunk of each block's keys.
//
// Roles (512 threads; registers dealt out by setmaxnreg, 176, 72 and 88 a thread):
//   warps 0..3, 4..7 : softmax of tile 0, of tile 1: thread r = query row r = TMEM lane r
//   warps 8..11      : outputs of both tiles (O / l -> bf16, or an fp32 partial); values that
//                      must not be multiplied as they are
//   warps 12, 13     : products of tile 0, of tile 1
//   warp 14          : TMA loads
//   warp 15          : the block's next item of work (up to two tiles of query rows of one
//                      sequence and key head), found from the lengths
//
// Values of keys that a row does not see have weight 0, but 0 times what is not finite
// is NaN.  Tiles with keys that some row of the block does not see (an item's last, at most
// three) therefore pass through the output warps before products may read them: what
// lies behind the sequence's end becomes zeros, and in what some rows see and others do not, values
// that are not finite do; they are then added to the outputs of the rows that see
// them.  (By the softmax warps, beside their scores: each tile's products then wait for both
// tiles' softmax there; 61 short prompts 283 us, by the output warps 275.)
//
// What bounds it.  A tile's chain: scores complete, softmax 0.55 us, p.v and the next q.k issued
// behind it, 1280 (192 columns) or 1024 cycles, and three signals of 0.1 us.  The two tiles'
// chains overlap, so that the tensor cores are busy 75 to 85 % of the time on long
// items; an item's start and end cost about 2 us (first loads, both chains in step).
// Measured in the first 0.1 s of calls, and after a second of them, when the power limit has lowered the
// clock: 76 heads of 4096 tokens over 4096 keys, no mask, 461 and 501 us = 1.77 and 1.63 PFLOP/s (93 % of the
// burst matrix rate, 97 % of the sustained one); one causal prompt of 16 heads of 16384 tokens 774 and 825 us =
// 1.78 and 1.67; two of 128 heads of 2048 and 4096 532 and 594 us = 1.62 and 1.45; 61 of 1 to 601 tokens, 64 heads, 278
// and 296 us = 4.9 and 4.6 TB/s; a single tile 6.2 us.
// On the way here (16384 tokens): one lane walking the products' loop 1841 us, all lanes 1476,
// whole boxes for two chunks and no row maxima 1288, a warp for each tile's products and code that fits
// the instruction cache 1132, loads and descriptors off the way 997 and 935, without the
// second sum 868, keys and values towards L2 820.  Not kept: P handed over by halves (930 where it was 895; the
// ragged 61 and chunks of a prompt gained 3 %), the rounded probabilities' sum (5 to 8 % more everywhere), queries,
// first keys and values towards L2 ahead of their item (61 short prompts 274 -> 276 to 281), both tiles on one
// tile's rows where rows are few, the products' loop flattened across items (64 on 8 heads 125 -> 155), four
// items in hand (137 -> 144), a third tile of queries instead of half a tile of ring for 128 columns (76 heads
// 405 -> 390, but 32 on 8 heads, causal, 331 -> 340), boxes of 64 tokens where a tile's last half is not
// needed (61 short prompts 274 -> 291, whose surplus of 190 MB read they would have halved).
//
// Waits are bounded; after one has run out every role leaves, and the block pauses
// before it frees TMEM and ends.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstddef>

#include "mla_decode.h"
#include "mla_internal.h"
#include "mla_ptx.cuh"

namespace mla {
namespace prefill {

constexpr int kThreads = 512;
constexpr int kRows = 128;    // query rows of a tile
constexpr int kKeys = 128;    // keys of a tile
constexpr int kNope = 128, kRope = 64, kValue = 128;
constexpr int kChunk = 16384; // [128 tokens x 64 columns] bf16
constexpr int kSmemData = 14 * kChunk;
constexpr int kItems = 2;     // the one that is worked on, and the next
constexpr uint32_t kBeside = 8;  // blocks of a head's query rows whose items follow each other
constexpr int kLead = 2;      // key tiles of an item still to be loaded when the next is looked for
constexpr int kDepth = 4;     // barriers of each kind: more tiles than the ring holds parts of
// Probabilities are taken against a reference 2^24 above the score of a piece's first key, and
// above the row's maximum from where a tile's probabilities sum past 1 on.  It need not be
// near the maximum: bf16 has fp32's exponents, so probabilities keep their precision
// wherever they lie.  So the maximum is hardly ever looked for and O hardly ever rescaled.
// r * sc + 24 is rounded to fp32, past kFar by more than 1: the weights of a row's largest scores could then
// leave fp32 at either end.  A row whose reference lies past kFar (a far row; no trained model has such
// scores) keeps r itself, in the scores' units: each tile's maximum goes into it, and it is subtracted from the tile's
// scores in TMEM before they are scaled.
constexpr float kAbove = 24.f, kMoveSum = 1.f, kFar = 16777216.f;
constexpr uint32_t kIdesc128 = idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdescPv = idesc_bf16(128, 128, false, true);
constexpr uint32_t kIdescPvHalf = idesc_bf16(128, 64, false, true);
// TMEM columns
constexpr uint32_t kColS = 0, kColO = 256;

struct Params {
  const int32_t* cu_q;   // [batch + 1]
  const int32_t* cu_k;
  int batch, total_q, total_k;
  uint32_t h_k;          // key heads
  int group;             // query heads of each
  int tokens;            // tokens of a tile: 128 / group
  uint64_t per_inverse;  // 2^38 / (2 * tokens), rounded up: quotients of up to 2^26 by it
  int causal;
  int rope_per_head;     // k_rope has a head dimension
  int splits;            // pieces that a row's keys are cut into, at most
  uint32_t parts;        // SMs
  float scale_log2;      // softmax_scale * log2 e
  __nv_bfloat16* out;
  int64_t out_token, out_head;  // strides in elements
  int out_wide;          // rows of out begin on 32 bytes
  float* lse;            // [h_q, total_q]
  float* ws_o;           // splits > 1: [splits, total_q, h_q, 128]
  float* ws_lse;         // [splits, h_q, total_q]
  const __nv_bfloat16* v;
  int64_t v_token, v_head;
  uint32_t* err;
};

struct Maps {
  CUtensorMap q, k, rope, v;  // boxes of one chunk of query rows, both chunks of keys, of position columns, of values
  CUtensorMap k1, v1;         // one chunk of keys, of values: where both would run past the ring's end
};

// One piece of work: up to two tiles of query rows of one sequence and key head, and
// the key tiles [first, first + n) of each.
struct Item {
  int32_t q_row;      // first token (of the packed rows)
  int32_t n_tok;      // tokens, at most 2 * Params::tokens; 0: no more work
  int32_t seen0;      // keys that the first token sees; one more per token up to k_len (causal)
  int32_t k_row;      // the sequence's first key (of the packed rows)
  int32_t k_len;
  int32_t head;       // key head
  int32_t split;
  int32_t first;      // first key tile
  int32_t n[2];       // key tiles of each tile of query rows
  int32_t off[2];     // each one's first token (n_tok or more: it has none)
  int32_t ahead;      // the block of rows with the most keys: it sends for them first
  uint32_t odd;       // a value that is not finite was taken out
};

struct Shared {
  alignas(16) uint4 answer;  // of a request to cancel a block
  uint64_t answered;
  uint64_t k_full[kDepth], k_empty[kDepth], v_full[kDepth], v_empty[kDepth];  // of a key tile's chunks
  uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2], o_full[2], o_free[2], sums_full[2], sums_free[2];
  uint64_t item_full[kItems], item_empty[kItems], item_ahead;
  uint64_t edge[kDepth];
  Item items[kItems];
  uint32_t tmem;
  volatile uint32_t busy[2];  // that tile's products are being issued
  uint32_t abort;
  float inv[2][kRows];  // 1 / (sum of a row's probabilities); 0 for a row that sees no key
};
constexpr int kSmemBytes = kSmemData + 1024 /* alignment */ + static_cast<int>(sizeof(Shared));
static_assert(kSmemBytes <= 232448, "shared memory of a block");

__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// mbar_wait in few instructions: the roles' code together has to stay within the
// instruction cache.  A wait that has run out sets *abort; the block reports it at its end.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  uint32_t t0 = 0;
  while (!mbar_try_wait(bar, parity)) {
    uint32_t now;
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(now));
    if (t0 == 0) t0 = now | 1u;
    if (now - t0 > static_cast<uint32_t>(kWaitTimeoutNs) && static_cast<int32_t>(now - t0) != -1) *abort = 1u;
    if (*abort) return false;
  }
  return true;
}

__device__ __forceinline__ void mbar_arrive_many(uint32_t bar, uint32_t count) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0], %1; }" ::"r"(bar), "r"(count) : "memory");
}

// Keys that token `at` of an item sees.
__device__ __forceinline__ int seen_by(const Item& it, int at, int causal) {
  if (!causal) return it.k_len;
  const int n = it.seen0 + at;
  return n < 0 ? 0 : (n > it.k_len ? it.k_len : n);
}

// Whether some row of the item does not see a key of tile t (of the sequence's).
__device__ __forceinline__ bool edge_tile(const Item& it, int t, int causal) {
  return (t + 1) * kKeys > seen_by(it, 0, causal);
}

// Reports sequences that do not follow each other within the tensors' rows.
__device__ __forceinline__ void check_ranges(const Params& p, int lane) {
  bool bad = false;
  for (int i = lane; i < p.batch; i += 32) {
    const int q0 = p.cu_q[i], q1 = p.cu_q[i + 1], k0 = p.cu_k[i], k1 = p.cu_k[i + 1];
    bad = bad || q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k;
  }
  if (bad && p.err) atomicOr(p.err, MLA_DEVERR_BAD_RANGE);
}

// Where a search for items stands: 32 sequences, a lane each, the one with the most keys
// first where the order counts, and the items before them.
struct Window {
  int base;                 // the first of the sequences; -1: none looked at
  uint32_t before, all;     // items of sequences before these, of these
  int q0, q_len, k0, k_len; // of the lane's sequence
  uint32_t blocks, mine, upto;  // its blocks of query rows, its items, those up to its last
  uint32_t heads;           // of a group of its
};

__device__ __forceinline__ void look_at(const Params& p, Window& w, int base, uint32_t before, int lane) {
  w.base = base;
  w.before = before;
  const int i = base + lane;
  int q0 = 0, q_len = 0, k0 = 0, k_len = 0;
  if (i < p.batch) {  // (clamped to rows that exist)
    q0 = min(max(p.cu_q[i], 0), p.total_q);
    q_len = min(max(p.cu_q[i + 1], q0), p.total_q) - q0;
    k0 = min(max(p.cu_k[i], 0), p.total_k);
    k_len = min(max(p.cu_k[i + 1], k0), p.total_k) - k0;
  }
  const int per = 2 * p.tokens;
  w.blocks = static_cast<uint32_t>(static_cast<uint64_t>(q_len + per - 1) * p.per_inverse >> 38);
  w.all = __reduce_add_sync(0xffffffffu, w.blocks) * (p.h_k * p.splits);
  // The order counts where items wait for an SM, differ in length, and the longest takes more than a
  // sixteenth of the call.  Otherwise sequences come as they lie: what boxes hold of the next
  // sequence's rows is then still in L2 when its turn comes (100 of 1 to 300 tokens, 128 heads, 483 us
  // sorted, 469 so; with an eighth 8 of 300 to 3000, 32 heads, 213 -> 225).
  const uint32_t tiles = static_cast<uint32_t>(k_len + kKeys - 1) / kKeys;
  int from = lane;
  const uint32_t most = __reduce_max_sync(0xffffffffu, w.blocks > 0 ? tiles : 0u);
  if (w.all > p.parts && most != __reduce_min_sync(0xffffffffu, w.blocks > 0 ? tiles : ~0u) &&
      static_cast<float>(most) * p.parts * 16.f > static_cast<float>(p.h_k) * __reduce_add_sync(0xffffffffu, w.blocks * tiles)) {
    int rank = 0;
#pragma unroll 1
    for (int o = 0; o < 32; ++o) {
      const int other = __shfl_sync(0xffffffffu, k_len, o);
      rank += other > k_len || (other == k_len && o < lane);
    }
#pragma unroll 1
    for (int o = 0; o < 32; ++o)
      if (__shfl_sync(0xffffffffu, rank, o) == lane) from = o;
  }
  w.q0 = __shfl_sync(0xffffffffu, q0, from);
  w.q_len = __shfl_sync(0xffffffffu, q_len, from);
  w.k0 = __shfl_sync(0xffffffffu, k0, from);
  w.k_len = __shfl_sync(0xffffffffu, k_len, from);
  w.blocks = __shfl_sync(0xffffffffu, w.blocks, from);
  w.mine = w.upto = w.blocks * (p.h_k * p.splits);
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, w.upto, o);
    if (lane >= o) w.upto += v;
  }
  w.heads = w.blocks * p.h_k <= 2 * p.parts ? p.h_k : max(2 * p.parts / w.blocks, 1u);
}

// Finds item `index` of the call (lanes of one warp together).  A sequence's items lie by
// groups of heads, as many as fill the device twice (their keys and values, some 40 MB whatever
// the length, stay in L2 meanwhile); in a group blocks of query rows come from the last, which
// has the most keys, to the first, eight of a head beside each other, and a block's splits.  (With a
// head's blocks apart, all heads' between them, each read its keys from memory: 2 requests of 1024 tokens over 4000
// and 8000 keys, 128 heads, 766 us, by twos 732, fours 661, eights 658, sixteens 657.)  Rows of an
// item that fill one tile only are tile 0 or 1 by turns: the next item's products and softmax then
// run beside it.
__device__ __forceinline__ bool find_item(const Params& p, uint32_t index, Window& w, Item& out, uint32_t turn, int lane) {
  if (w.base < 0 || index < w.before) {
    w.base = -32;
    w.before = w.all = 0u;
  }
#pragma unroll 1
  while (index - w.before >= w.all) {
    if (w.base + 32 >= p.batch) return false;
    look_at(p, w, w.base + 32, w.before + w.all, lane);
  }
  const uint32_t local = index - (w.before + w.upto - w.mine);  // within the lane's sequence, if below its items
  const uint32_t hit = __ballot_sync(0xffffffffu, local < w.mine);
  if (hit == 0u) return false;  // (sequences that overlap beyond 32 bits of items)
  if (lane == __ffs(hit) - 1) {
    const uint32_t blocks = w.blocks;
    // (most calls have a group or a piece; divisions take as long as a load)
    const uint32_t first_head = w.heads >= p.h_k ? 0u : local / (w.heads * blocks * p.splits) * w.heads;
    const uint32_t here = min(w.heads, p.h_k - first_head);  // (the last group may be smaller)
    const uint32_t rem = local - first_head * blocks * p.splits, by_split = p.splits == 1 ? rem : rem / p.splits;
    const uint32_t from = blocks <= kBeside ? 0u : by_split / (here * kBeside) * kBeside;
    const uint32_t in = by_split - here * from, beside = min(blocks - from, kBeside), hd = in / beside, row = from + in - hd * beside;
    const int split = rem - by_split * p.splits, head = first_head + hd, block = blocks - 1 - row;
    const int per = 2 * p.tokens, at = block * per;
    Item it;
    it.q_row = w.q0 + at;
    it.n_tok = min(w.q_len - at, per);
    it.k_row = w.k0;
    it.k_len = w.k_len;
    it.seen0 = w.k_len - w.q_len + at + 1;
    it.head = head;
    it.split = split;
    it.off[0] = it.n_tok <= p.tokens && turn != 0 ? p.tokens : 0;
    it.off[1] = it.n_tok <= p.tokens && turn != 0 ? 0 : p.tokens;
    int tiles[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int last = min(it.n_tok, it.off[x] + p.tokens) - 1;  // the tile's last token
      tiles[x] = last >= it.off[x] ? (seen_by(it, last, p.causal) + kKeys - 1) / kKeys : 0;
    }
    const int most = max(tiles[0], tiles[1]);
    it.first = p.splits == 1 ? 0 : most * split / p.splits;  // (2^18 tiles, 2^5 splits at most)
    const int end = p.splits == 1 ? most : most * (split + 1) / p.splits;
#pragma unroll
    for (int x = 0; x < 2; ++x) it.n[x] = max(min(tiles[x], end) - it.first, 0);
    it.ahead = row == 0 && p.splits == 1;
    it.odd = 0u;
    out = it;
  }
  return true;
}

// 32 bytes, a whole sector, by one thread.
__device__ __forceinline__ void st_global_v8(void* to, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// One 32-bit column: thread i gets lane (base + i).
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(taddr));
  return __uint_as_float(r);
}

// Zeros what is not finite in a unit of eight values in shared memory; whether there was any.
__device__ __forceinline__ bool take_out(uint32_t addr) {
  const uint4 v = ld_shared_v4(addr);
  const uint4 w = make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z), finite_bf16x2(v.w));
  const bool any = ((v.x ^ w.x) | (v.y ^ w.y) | (v.z ^ w.z) | (v.w ^ w.w)) != 0u;
  if (any) st_shared_v4(addr, w.x, w.y, w.z, w.w);
  return any;
}

// x * 0 + acc for two bf16: NaN from the first value that is not finite on.
__device__ __forceinline__ uint32_t note_odd(uint32_t x, uint32_t acc) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(acc));
  return r;
}

// One chunk of a value tile before products read it, by four warps: rows from `valid` on
// become zeros; in rows `seen` .. valid - 1, which some query rows see and others do not,
// values that are not finite do.  Returns whether the warp found any.  A row's eight
// 16-byte units lie swizzled within its 128 bytes, so units are taken as they come;
// each thread has eight of the chunk's 1024.
__device__ __forceinline__ bool fix_values(uint32_t at, int seen, int valid, int thread) {
  uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ld_shared_v4(at + 16 * (thread + 128 * (4 * h + i)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = thread + 128 * (4 * h + i);
      if (u >= valid * 8)
        st_shared_v4(at + 16 * u, 0u, 0u, 0u, 0u);
      else
        acc[i] = note_odd(v[i].w, note_odd(v[i].z, note_odd(v[i].y, note_odd(v[i].x, acc[i]))));
    }
  }
  bool odd = false;
  if (__any_sync(0xffffffffu, ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7F807F80u) != 0u)) {  // (sums of zeros otherwise)
#pragma unroll 1
    for (int u = thread; u < valid * 8; u += 128)
      if (u >= seen * 8) odd |= take_out(at + 16 * u);
  }
  return __any_sync(0xffffffffu, odd);
}

// One lane of the warp, the same whenever the whole warp asks.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred e; elect.sync _|e, 0xffffffff; selp.u32 %0, 1, 0, e; }" : "=r"(r));
  return r;
}
// Shared-memory operands (128-byte swizzle, 8-row groups 1024 bytes apart) by the lower
// half of their descriptors; the upper is the same for all of them.
constexpr uint32_t kDescHi = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | (lbo >> 4 << 16); }
// The same value in every lane, known to be so.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
// Products and commits by the lane whose `leader` is set, in code that all lanes run.
__device__ __forceinline__ void mma_ss_if(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, q; .reg .b64 a, b; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; mov.b64 a, {%1, %6}; mov.b64 b, {%2, %6};"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p; }" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(leader),
      "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p, q; .reg .b64 b; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0; mov.b64 b, {%2, %6};"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p; }" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(leader),
      "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0;"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar), "r"(leader)
      : "memory");
}

// A box towards L2.
__device__ __forceinline__ void prefetch_4d_if(uint32_t leader, const void* tmap, int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile("{ .reg .pred q; setp.ne.b32 q, %5, 0; @q cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}]; }" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(leader)
               : "memory");
}

// Asks for a block of this grid that has not begun not to begin: 16 bytes of answer at
// `answer`, completing on `bar`.
__device__ __forceinline__ void cancel_a_block(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer), "r"(bar)
               : "memory");
}
// Whether a block was cancelled, and its index.
__device__ __forceinline__ bool cancelled_block(uint32_t answer, uint32_t* index) {
  uint32_t got, x;
  asm volatile(
      "{ .reg .pred p; .reg .b128 r; ld.shared.b128 r, [%2]; clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;"
      " selp.u32 %1, 1, 0, p; mov.u32 %0, 0; @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r; }"
      : "=r"(x), "=r"(got) : "r"(answer) : "memory");
  if (got) *index = x;
  return got != 0u;
}

// Loads of one box, and the arrival that expects their bytes, by the lane whose `leader` is set.
__device__ __forceinline__ void expect_if(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{ .reg .pred q; .reg .b64 st; setp.ne.b32 q, %2, 0; @q mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void load_4d_if(uint32_t leader, uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z, int32_t w,
                                           uint32_t bar, uint64_t policy) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %8, 0;"
      " @q cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7; }" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void load_5d_if(uint32_t leader, uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z, int32_t w,
                                           int32_t v, uint32_t bar, uint64_t policy) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %9, 0;"
      " @q cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8; }" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(bar), "l"(policy), "r"(leader)
      : "memory");
}

// kHasRope: 192 columns of q and k (three chunks a key tile, a ring of 8), else 128
// (two chunks, a ring of 10).
template <bool kHasRope>
__global__ void __launch_bounds__(kThreads, 1)
    mla_prefill_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  constexpr int kQk = kHasRope ? 3 : 2;    // chunks of a tile's keys
  constexpr int kPer = kQk + 2;            // of its keys and values
  constexpr int kRing = 14 - 2 * kQk;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_base = base, ring = base + 2 * kQk * kChunk;
  Shared* sm = reinterpret_cast<Shared*>(smem_raw + (base - smem_u32(smem_raw)) + kSmemData);
  volatile uint32_t* abort_flag = &sm->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto bar = [](uint64_t& b) { return smem_u32(&b); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kDepth; ++i) {
      mbar_init(bar(sm->k_full[i]), 1);
      mbar_init(bar(sm->k_empty[i]), 2);
      mbar_init(bar(sm->v_full[i]), 4);  // a load's arrival and three more, or four warps'
      mbar_init(bar(sm->v_empty[i]), 2);
      mbar_init(bar(sm->edge[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sm->q_full[i]), 1);
      mbar_init(bar(sm->q_empty[i]), 1);
      mbar_init(bar(sm->s_full[i]), 1);
      mbar_init(bar(sm->p_ready[i]), 4);
      mbar_init(bar(sm->o_full[i]), 1);
      mbar_init(bar(sm->o_free[i]), 4);
      mbar_init(bar(sm->sums_full[i]), 4);
      mbar_init(bar(sm->sums_free[i]), 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar(sm->item_full[i]), 1);
      mbar_init(bar(sm->item_empty[i]), 15);  // all warps but the one that fills them
    }
    mbar_init(bar(sm->answered), 1);
    mbar_init(bar(sm->item_ahead), 1);
    sm->busy[0] = sm->busy[1] = 0u;
    sm->abort = 0u;
    fence_mbarrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
    if (kHasRope) {
      tma_prefetch_desc(&maps.rope);
      tma_prefetch_desc(&maps.k1);
      tma_prefetch_desc(&maps.v1);
    }
  }
  if (warp == 12) tmem_alloc(smem_u32(&sm->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;
  pdl_launch_dependents();
  pdl_wait_primary();

  // The next item for this role, or false: no more (or an abort).  All lanes of a warp.
  uint32_t it_n = 0;
  const Item* it = sm->items;
  auto next_item = [&]() -> bool {
    const uint32_t slot = it_n % kItems;
    bool ok = wait_for(bar(sm->item_full[slot]), (it_n / kItems) & 1, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return false;
    it = &sm->items[slot];
    return it->n_tok > 0;
  };
  auto done_item = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(sm->item_empty[it_n % kItems]));
    ++it_n;
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2, r = threadIdx.x & 127;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    const uint32_t t_s = t_lane + kColS + 128 * x, t_o = t_lane + kColO + 128 * x;
    const int my_tok = r / p.group, my_sub = r % p.group;
    const float sc = p.scale_log2;
    uint32_t tiles = 0, items = 0;
    bool ok = true;
    while (ok && next_item()) {
      const int n = it->n[x];
      const int at = it->off[x] + my_tok;
      const int seen = seen_by(*it, min(at, it->n_tok - 1), p.causal);
      const bool row = my_tok < p.tokens && at < it->n_tok;
      float m = 0.f, lsum = 0.f;
      bool far = false, any_far = false;  // this row, some row of the warp
      float far_ref = -INFINITY;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int t = it->first + i;
        const bool edge = edge_tile(*it, t, p.causal);
        wait_for(bar(sm->s_full[x]), tiles++ & 1, abort_flag);  // (after an abort the item runs out without waiting)
        __syncwarp();
        tc_fence_after();
        const int lim = seen - t * kKeys;
        float l[4][2];  // (one chain of additions would take as long as the exponentials)
        uint32_t pk[4][16];
        // A tile with unseen keys: their scores become -inf in TMEM before the pass reads them,
        // by blocks of 32 keys from the first that not all of the warp's rows see.
        if (edge) {
#pragma unroll 1
          for (int j = max(__reduce_min_sync(0xffffffffu, lim), 0) / 32; j < 4; ++j) {
            float v[32];
            tmem_ld32(t_s + 32 * j, v);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = k < lim - 32 * j ? v[k] : -INFINITY;
            tmem_st32(t_s + 32 * j, v);
          }
          tmem_wait_st();
        }
        // (a row that does not see the piece's first key sees none of it; where that key's score is no reference, the
        // sum is NaN and the pass taken again)
        if (i == 0) {
          m = tmem_ld1(t_s) * sc + kAbove;
          m = lim <= 0 ? 0.f : (fabsf(m) <= kFar ? m : NAN);
        }
        // The row maximum is looked for only where the probabilities sum past the bound, which one of
        // them far above the reference needs; the warp then takes the pass again.
        bool again = false;
#pragma unroll 1
        do {
          if (again || any_far) {
            float top = -INFINITY;
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
              float v[16];
              tmem_ld16(t_s + 16 * j, v);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; k += 2) top = fmax3(top, v[k], v[k + 1]);
            }
            // (this tile's scores were issued after the last tile's p.v and have completed: O holds every tile
            // before; a row moves by its own sum alone, whatever its neighbours in the warp do)
            float alpha = 1.f, less = 0.f;  // less: to be subtracted from the row's scores
            if (far && !again) {
              if (top > far_ref) {
                alpha = fast_exp2((far_ref - top) * sc);
                far_ref = top;
              }
              less = far_ref == -INFINITY ? 0.f : far_ref;
            } else if (!far && again) {
              const float up = top * sc + kAbove;
              if (!(l[0][0] <= kMoveSum) && !(up <= m)) {
                far = row && !(fabsf(up) <= kFar);
                if (i > 0) alpha = fast_exp2(far ? __fmaf_rn(-top, sc, m) - kAbove : m - up);
                m = far ? kAbove : up;
                if (far) far_ref = top;
                if (far && top != -INFINITY) less = top;
              }
            }
            lsum *= alpha;
#pragma unroll 1
            for (int j = 0; j < 8 && i > 0; ++j) {
              float o[16];
              tmem_ld16(t_o + 16 * j, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= alpha;
              tmem_st16(t_o + 16 * j, o);
            }
            any_far = __any_sync(0xffffffffu, far);
            if (any_far) {
#pragma unroll 1
              for (int j = 0; j < 8; ++j) {
                float v[16];
                tmem_ld16(t_s + 16 * j, v);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] -= less;
                tmem_st16(t_s + 16 * j, v);
              }
              tmem_wait_st();
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) l[j][0] = l[j][1] = 0.f;
          float s[2][32];  // 32 scores on their way while 32 are worked on
          tmem_ld32(t_s, s[0]);
          tmem_wait_ld();
          const float neg_m = -m;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j < 3) tmem_ld32(t_s + 32 * (j + 1), s[(j + 1) & 1]);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x0, x1;
              asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %4}; mov.b64 c, {%5, %5};"
                  " fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d; }"
                  : "=f"(x0), "=f"(x1) : "f"(s[j & 1][2 * k]), "f"(s[j & 1][2 * k + 1]), "f"(sc), "f"(neg_m));
              const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
              pk[j][k] = pack_bf16x2(e0, e1);
              asm("{ .reg .b64 a, b, c; mov.b64 a, {%0, %1}; mov.b64 b, {%2, %3}; add.rn.f32x2 c, a, b; mov.b64 {%0, %1}, c; }"
                  : "+f"(l[k & 3][0]), "+f"(l[k & 3][1]) : "f"(e0), "f"(e1));
            }
            if (j < 3) tmem_wait_ld();
          }
          l[0][0] = (l[0][0] + l[0][1]) + (l[1][0] + l[1][1]) + ((l[2][0] + l[2][1]) + (l[3][0] + l[3][1]));
          again = !again && __any_sync(0xffffffffu, row && !(l[0][0] <= kMoveSum));
        } while (again);
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_st16u(t_s + 16 * j, pk[j]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm->p_ready[x]));
        lsum += l[0][0];
      }
      if (n > 0) {
        const bool has = !(lsum <= 0.f);  // (NaN: a key that is not finite, no empty row)
        if (row) {
          const int64_t h = static_cast<int64_t>(it->head) * p.group + my_sub, tok = it->q_row + at;
          constexpr float kLn2 = 0.69314718055994531f;
          const float l2 = (m + __log2f(lsum)) * kLn2, l = !has ? -INFINITY : (far ? __fmaf_rn(far_ref, sc * kLn2, l2) : l2);
          if (p.splits == 1)
            p.lse[h * p.total_q + tok] = l;
          else
            p.ws_lse[(it->split * static_cast<int64_t>(p.h_k) * p.group + h) * p.total_q + tok] = l;
        }
        ok = wait_for(bar(sm->sums_free[x]), (items & 1) ^ 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        sm->inv[x][r] = has ? __frcp_rn(lsum) : 0.f;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm->sums_full[x]));
        ++items;
      }
      done_item();
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ------------------------------------------------------------ outputs
    const int r = threadIdx.x & 127;
    const int my_tok = r / p.group, my_sub = r % p.group;
    uint32_t items[2] = {0u, 0u}, tile = 0, edges = 0;
    bool ok = true;
    while (ok && next_item()) {
      // The item's tiles with unseen keys, which are its last; then its rows.
      const int n = max(it->n[0], it->n[1]), low = seen_by(*it, 0, p.causal);
#pragma unroll 1
      for (int i = max(low / kKeys - it->first, 0); i < n; ++i, ++edges) {
        ok = __all_sync(0xffffffffu, wait_for(bar(sm->edge[edges % kDepth]), (edges / kDepth) & 1, abort_flag));
        if (!ok) break;
        const int from = (it->first + i) * kKeys, seen = max(0, low - from), valid = min(kKeys, it->k_len - from);
        bool odd = false;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) odd |= fix_values(ring + ((tile + i) * kPer + kQk + c) % kRing * kChunk, seen, valid, r);
        if (odd) *reinterpret_cast<volatile uint32_t*>(&sm->items[it_n % kItems].odd) = 1u;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm->v_full[(tile + i) % kDepth]));
      }
      tile += n;
#pragma unroll 1
      for (int x = 0; x < 2 && ok; ++x) {
        const int at = it->off[x] + my_tok;
        const bool row = my_tok < p.tokens && at < it->n_tok;
        const int64_t h = static_cast<int64_t>(it->head) * p.group + my_sub, tok = it->q_row + at;
        const int64_t part = (static_cast<int64_t>(it->split) * p.total_q + tok) * p.h_k * p.group + h;
        uint4* dst = reinterpret_cast<uint4*>(p.out + tok * p.out_token + h * p.out_head);
        float4* ws = reinterpret_cast<float4*>(p.ws_o + part * kValue);
        float inv = 0.f;
        if (it->n[x] > 0) {
          const uint32_t par = items[x] & 1;
          ++items[x];
          ok = wait_for(bar(sm->sums_full[x]), par, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          inv = sm->inv[x][r];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sm->sums_free[x]));
          ok = wait_for(bar(sm->o_full[x]), par, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        } else if (row) {  // no key: the softmax warps have nothing to say
          if (p.splits == 1)
            p.lse[h * p.total_q + tok] = -INFINITY;
          else
            p.ws_lse[(static_cast<int64_t>(it->split) * p.h_k * p.group + h) * p.total_q + tok] = -INFINITY;
        }
        const uint32_t t_o = tmem + (static_cast<uint32_t>(warp & 3) << 21) + kColO + 128 * x;
        auto freed = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sm->o_free[x]));
        };
        if (it->n[x] > 0 && p.splits == 1) {
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            float o[32];
            tmem_ld32(t_o + 32 * j, o);
            tmem_wait_ld();
            uint32_t w[2][8];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k / 8][k % 8] = inv != 0.f ? pack_bf16x2(o[2 * k] * inv, o[2 * k + 1] * inv) : 0u;
            if (row && p.out_wide) {
              st_global_v8(dst + 4 * j, w[0]);
              st_global_v8(dst + 4 * j + 2, w[1]);
            } else if (row) {
#pragma unroll
              for (int k = 0; k < 4; ++k) dst[4 * j + k] = make_uint4(w[k / 2][4 * (k & 1)], w[k / 2][4 * (k & 1) + 1], w[k / 2][4 * (k & 1) + 2], w[k / 2][4 * (k & 1) + 3]);
            }
          }
          freed();
        } else if (it->n[x] > 0) {
#pragma unroll 1
          for (int j = 0; j < 8; ++j) {
            float o[16];
            tmem_ld16(t_o + 16 * j, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = inv != 0.f ? o[k] * inv : 0.f;
            if (row) {
#pragma unroll
              for (int k = 0; k < 2; ++k) st_global_v8(ws + 4 * j + 2 * k, reinterpret_cast<const uint32_t(&)[8]>(o[8 * k]));
            }
          }
          freed();
        } else if (row && p.splits == 1) {  // (a partial row with an lse of -inf has no weight, whatever it holds)
#pragma unroll 1
          for (int j = 0; j < 16; ++j) dst[j] = make_uint4(0u, 0u, 0u, 0u);
        }
        // what was taken out, onto the rows that see it (infinities and NaN: a sum of them, whatever their weights)
        if (it->n[x] > 0 && *reinterpret_cast<const volatile uint32_t*>(&it->odd) != 0u && row && inv != 0.f) {
          const int low = seen_by(*it, 0, p.causal), end = (it->first + it->n[x]) * kKeys, mine = seen_by(*it, at, p.causal);
          const int from = low > it->first * kKeys ? low : it->first * kKeys, upto = mine < end ? mine : end;
#pragma unroll 1
          for (int c = 0; c < kValue; ++c) {
            const __nv_bfloat16* v = p.v + static_cast<int64_t>(it->k_row + from) * p.v_token + it->head * p.v_head + c;
            float sum = 0.f;
#pragma unroll 1
            for (int t = from; t < upto; ++t, v += p.v_token) {
              const float f = __bfloat162float(*v);
              if (!(fabsf(f) < INFINITY)) sum += f;
            }
            if (sum == 0.f) continue;
            if (p.splits == 1) {
              __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(dst) + c;
              *o = __float2bfloat16(__bfloat162float(*o) + sum);
            } else {
              reinterpret_cast<float*>(ws)[c] += sum;
            }
          }
        }
      }
      if (!ok) break;
      done_item();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp < 14) {
      // ---------------------------------------------------------- products
      // A warp for each tile of query rows: while one waits or fetches descriptors the other's
      // products run (one warp for both left the tensor cores idle for a third of
      // the time).  All lanes walk the same path and one of them issues, so that descriptors
      // stay in uniform registers.  After an abort the loops run out without waiting.
      const int x = warp - 12;
      uint32_t tile = 0;                  // key tiles of all items so far
      uint32_t items = 0, tiles = 0;      // of this tile of rows
      const uint32_t leader = elect_one();
      const uint32_t a_q = uniform(desc_lo(q_base + x * kQk * kChunk, 16));
      const uint32_t d_s = uniform(tmem + kColS + 128 * x), d_o = uniform(tmem + kColO + 128 * x);
      auto wait = [&](uint64_t& b, uint32_t parity) { wait_for(bar(b), parity, abort_flag); };
      // Products of both tiles issued at the same time take turns and complete together: the tiles are in step
      // from then on, and the tensor cores idle while both are in softmax.  So whoever finds the
      // other at it lets it finish (no more than a hint: after a hundred looks it goes on).  64 on 8
      // heads of 128 columns 126.6 -> 120.2 us, 76 heads of 4096 keys without a mask 420 -> 409; 192 columns fall
      // out of step by themselves, and the looks, on the tiles' way, cost more (two prompts 528 -> 568).
      auto take_turn = [&]() {
#pragma unroll 1
        for (int k = 0; k < 100 && !kHasRope; ++k) {
          if (sm->busy[x ^ 1] != 0u) continue;
          sm->busy[x] = 1u;
          if (x == 0 || sm->busy[0] == 0u) break;
          sm->busy[1] = 0u;
        }
      };
      while (next_item()) {
        const int n = __reduce_max_sync(0xffffffffu, max(it->n[0], it->n[1])), mine = __reduce_max_sync(0xffffffffu, it->n[x]);
#pragma unroll 1
        for (int i = -1; i < n; ++i) {
          // O += P . V of tile i, and behind it S = Q . K^T of the next (S lies where P did).  All
          // that can be known before P is there is looked up before: the products then
          // follow one another.
          const uint32_t t = tile + i, o = t % kDepth, t1 = t + 1, o1 = t1 % kDepth;
          const bool pv = i >= 0 && i < mine, qk = i + 1 < mine;
          const uint32_t s0 = (t * kPer + kQk) % kRing, b_v = uniform(desc_lo(ring + s0 * kChunk, kChunk));
          uint32_t b_k[kQk];
#pragma unroll
          for (int c = 0; c < kQk; ++c) b_k[c] = uniform(desc_lo(ring + (t1 * kPer + c) % kRing * kChunk, 16));
          if (i == 0 && pv) wait(sm->o_free[x], (items & 1) ^ 1);
          if (i >= 0) wait(sm->v_full[o], (t / kDepth) & 1);
          if (i < 0 && qk) wait(sm->q_full[x], items & 1);
          if (!kHasRope && i + 1 < n) wait(sm->k_full[o1], (t1 / kDepth) & 1);
          if (pv) {
            wait(sm->p_ready[x], tiles & 1);
            ++tiles;
            take_turn();
            tc_fence_after();
            if (s0 + 1 < kRing) {
#pragma unroll
              for (int k = 0; k < 8; ++k) mma_ts_if(leader, d_o, d_s + 8 * k, b_v + 128 * k, kIdescPv, i > 0 || k != 0);
            } else {  // the chunks lie behind each other but where the ring ends
              const uint32_t b1 = uniform(desc_lo(ring, kChunk));
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                mma_ts_if(leader, d_o, d_s + 8 * k, b_v + 128 * k, kIdescPvHalf, i > 0 || k != 0);
                mma_ts_if(leader, d_o + 64, d_s + 8 * k, b1 + 128 * k, kIdescPvHalf, i > 0 || k != 0);
              }
            }
            if (i == mine - 1) {
              commit_if(leader, bar(sm->o_full[x]));
              ++items;
            }
            commit_if(leader, bar(sm->v_empty[o]));
          }
          // (the ring of 192-wide keys holds 1.6 tiles: the next keys may still be on their way)
          if (kHasRope && i + 1 < n) wait(sm->k_full[o1], (t1 / kDepth) & 1);
          if (qk) {
            if (!pv) take_turn();
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kQk; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ss_if(leader, d_s, a_q + c * (kChunk / 16) + 2 * k, b_k[c] + 2 * k, kIdesc128, (c | k) != 0);
            commit_if(leader, bar(sm->s_full[x]));
            if (i + 2 == mine) commit_if(leader, bar(sm->q_empty[x]));
            commit_if(leader, bar(sm->k_empty[o1]));
          }
          if (!kHasRope) sm->busy[x] = 0u;
          // tiles that only the other rows have
          __syncwarp();
          if (lane == 0 && i >= 0 && !pv) mbar_arrive(bar(sm->v_empty[o]));
          if (lane == 0 && i + 1 < n && !qk) mbar_arrive(bar(sm->k_empty[o1]));
        }
        tile += n;
        done_item();
      }
    } else if (warp == 14) {
      // ------------------------------------------------------------- loads
      // A box costs its SM a fixed time besides its bytes: both chunks of keys, and of values,
      // come in one.  Like the products, in code that all lanes run.  A tile's keys take
      // the place of values kV tiles back (and of what lies before), its values that of keys kK tiles back.
      constexpr uint32_t kV = kHasRope ? 2 : 3, kK = kHasRope ? 1 : 2;
      uint32_t tile = 0, edges = 0, items[2] = {0u, 0u};
      const uint64_t keep = l2_policy_evict_last(), once = l2_policy_evict_first();
      const uint32_t leader = elect_one();
      bool ok = true;
      auto wait = [&](uint64_t& b, uint32_t parity) { return ok = __all_sync(0xffffffffu, wait_for(bar(b), parity, abort_flag)); };
      while (ok && next_item()) {
        const int n = __reduce_max_sync(0xffffffffu, max(it->n[0], it->n[1])), head = uniform(it->head);
        const int rope_head = p.rope_per_head ? head : 0;
        int row = uniform(it->k_row + it->first * kKeys);
        if (n <= kLead && lane == 0) mbar_arrive(bar(sm->item_ahead));
        auto queries = [&](int x) {
          if (it->n[x] == 0) return;
          if (!wait(sm->q_empty[x], (items[x]++ & 1) ^ 1)) return;
          expect_if(leader, bar(sm->q_full[x]), kQk * 128u * p.group * p.tokens);
          const int q_row = uniform(it->q_row + it->off[x]);
#pragma unroll
          for (int c = 0; c < kQk; ++c)
            load_5d_if(leader, q_base + (x * kQk + c) * kChunk, &maps.q, 0, 0, q_row, c, head, bar(sm->q_full[x]), once);
        };
        if (n > 0) queries(0);
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i, ++tile, row += kKeys) {
          const uint32_t c0 = uniform(tile * kPer % kRing), cv = (c0 + kQk) % kRing, o = tile % kDepth;
          if (tile >= kV && !wait(sm->v_empty[(tile - kV) % kDepth], ((tile - kV) / kDepth) & 1)) break;
          if (i + kLead == n && i > 0 && lane == 0) mbar_arrive(bar(sm->item_ahead));
          const uint32_t kb = uniform(bar(sm->k_full[o]));
          expect_if(leader, kb, kQk * kChunk);
          if (!kHasRope || c0 + 1 < kRing) {
            load_4d_if(leader, ring + c0 * kChunk, &maps.k, 0, row, 0, head, kb, keep);
          } else {  // (a pair that would run past the ring's end, by its chunks)
            load_4d_if(leader, ring + c0 * kChunk, &maps.k1, 0, row, 0, head, kb, keep);
            load_4d_if(leader, ring, &maps.k1, 0, row, 1, head, kb, keep);
          }
          if (kHasRope) load_4d_if(leader, ring + (c0 + 2) % kRing * kChunk, &maps.rope, 0, row, 0, rope_head, kb, keep);
          if (i == 0) queries(1);
          if (!ok || (tile >= kK && !wait(sm->k_empty[(tile - kK) % kDepth], ((tile - kK) / kDepth) & 1))) break;
          // values of a tile with unseen keys complete on a barrier of the output warps', which then complete the products'
          const bool edge = edge_tile(*it, it->first + i, p.causal);
          // the ring is short of a load's way from memory; of blocks on the same keys the longest sends
          // for them (one prompt of 16384 tokens 855 -> 820 us; pieces of a few rows' keys are
          // slower with it, 64 -> 67)
          if (it->ahead && i + 2 < n) {
            prefetch_4d_if(leader, &maps.k, 0, row + 2 * kKeys, 0, head);
            prefetch_4d_if(leader, &maps.v, 0, row + 1 * kKeys, 0, head);
          }
          const uint32_t vb = uniform(bar(edge ? sm->edge[edges++ % kDepth] : sm->v_full[o]));
          expect_if(leader, vb, 2 * kChunk);
          if (leader && !edge) mbar_arrive_many(vb, 3);
          if (!kHasRope || cv + 1 < kRing) {
            load_4d_if(leader, ring + cv * kChunk, &maps.v, 0, row, 0, head, vb, keep);
          } else {
            load_4d_if(leader, ring + cv * kChunk, &maps.v1, 0, row, 0, head, vb, keep);
            load_4d_if(leader, ring, &maps.v1, 0, row, 1, head, vb, keep);
          }
        }
        if (!ok) break;
        done_item();
      }
    } else {
      // ------------------------------------------------------------- items
      // The grid has a block for every item that the lengths allow.  A block that runs takes on,
      // when it is through with its own item, one whose block has not begun: that block is
      // cancelled and its index comes back.  So items go to whoever is free first, without a counter
      // in memory that calls would share.
      Window window;
      window.base = -1;
      uint32_t index = blockIdx.x, asked = 0;
      bool have = true, ok = true;
      for (uint32_t k = 0;; ++k) {
        Item* slot = &sm->items[k % kItems];
        ok = __all_sync(0xffffffffu, wait_for(bar(sm->item_empty[k % kItems]), ((k / kItems) & 1) ^ 1, abort_flag));
        // The next item is taken on when the last loads of the one before are due: early enough
        // for its own, and so late that nobody sits on work that others could begin (64 on 8
        // heads, three prompts: 134 us with an item in hand all the time, 125 so).
        if (k > 0) ok = ok && __all_sync(0xffffffffu, wait_for(bar(sm->item_ahead), (k - 1) & 1, abort_flag));
        bool found = false, first = false;
        while (ok && !found) {
          if (!have) {
            if (lane == 0) {
              fence_proxy_async_smem();  // the last answer has been read
              mbar_arrive_expect_tx(bar(sm->answered), 16);
              cancel_a_block(smem_u32(&sm->answer), bar(sm->answered));
            }
            ok = __all_sync(0xffffffffu, wait_for(bar(sm->answered), asked++ & 1, abort_flag));
            if (!ok || !cancelled_block(smem_u32(&sm->answer), &index)) break;  // (after a no, no further question)
          }
          have = false;
          first = first || index == 0u;  // (whether there is an item behind it or not)
          found = find_item(p, index, window, *slot, k & 1, lane);  // (the grid may have more blocks than items)
        }
        if (!ok) break;
        if (!found && lane == 0) slot->n_tok = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm->item_full[k % kItems]));
        if (first) check_ranges(p, lane);  // (by whoever has the first block, behind its item)
        if (!found) break;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, MLA_DEVERR_TIMEOUT);
    settle_after_abort();
  }
  if (warp == 12) {
    tc_fence_after();
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace prefill
}  // namespace mla
