// Split-KV MLA decode kernel for sm_103a (tcgen05 MMA, TMEM accumulators,
// TMA-fed shared-memory ring, warp-specialised roles).
//
// One CTA owns 64 query rows (the heads of one block of one query token) and
// walks the (sequence, 128-key tile) range its schedule part assigns.  Per
// tile it computes, transposed so that key tokens sit on TMEM lanes:
//
//   S^T[128 tokens x 64 rows]  = K_tile[128 x 576] . Q^T          (QK^T, K = 576)
//   online softmax over tokens (column-wise, fp32, warp shuffles)
//   O^T[512 x 64 rows]        += V_tile^T[512 x 128] . P^T[128 x 64] (PV)
//
// with V_tile = the first 512 columns of the same shared-memory tile, so each
// 576-wide cached row is loaded once and feeds both products (FlashMLA deep
// dive, "Theoretical Analysis": K and V are the same latent row).  The TMEM
// accumulators hold O^T (4 x 64 columns) and S^T (64 columns); no output
// matrix lives in registers, which is why no seesaw schedule is needed here
// (the seesaw in the FlashMLA deep dive exists because WGMMA keeps O in
// registers).
//
// Roles (576 threads; 96 registers per thread: five warps share each of two
// SM sub-partitions):
//   warps 0..15    : four softmax warpgroups, query rows 16g .. 16g+15 each;
//                    FP8 cache: before each tile's scores they also convert
//                    the staged codes to bf16 in place (one 16-code unit per
//                    thread per chunk)
//   warp 16        : producer (lane 0; sparse: all lanes gather): TMA loads of
//                    Q (once per piece) and of each tile's 9 column chunks
//                    (two 64-token pages per chunk); FP8 cache: the raw codes
//                    and scales of the latent chunks (staged inside their
//                    slots) and the bf16 RoPE chunk, and with two head blocks
//                    the copy of every converted chunk into the peer CTA
//   warp 17        : TMEM allocation; lane 0 issues every MMA
//
// Shared memory (1024-byte aligned): 9 KV chunk slots of [128 tok x 64 col]
// bf16 (16 KB each, 128-byte swizzle), Q as 9 chunks of [64 rows x 64 col]
// (8 KB each).  Slot 8 (the RoPE columns) is dead after QK^T and holds P^T
// during PV.
//
// Windowed attention (kWindow, mla_window.cuh) runs the same loop over pieces
// that one warp works out, with several tokens of a request in the 64 rows when
// heads are few.  64 heads: 150 requests over 4000 keys take 158 us from the bf16
// cache (4.5 TB/s, 67 % of the copy rate: shared memory holds one tile, whose chunks
// are requested one by one as P.V of the tile before frees them), 230 us from the
// 656-byte cache and 226 us from the 528-byte one: there a tile's chain bounds it -
// slots free, codes arrive, eight chunks converted, scores, softmax, P.V - at 6.9 us
// a tile, of which the conversion's arithmetic is 1.2.  Rejected (from 233 us): two or four chunks converted
// between barriers (229 and 260 us; two head blocks 575 -> 612 and 685), scales
// fetched once a tile (239), output rows in 16-byte pieces by lane exchanges
// (64 requests over 128 keys 17.4 -> 18.9 us).
//
// Waits are bounded (mbar_wait*).  After an abort the producers and the MMA thread
// leave their loops; softmax warps leave together (FP8 caches, by a vote) or go on
// to the end without waiting and without writing; the work list is walked out, and
// the block pauses for what is still in flight before it ends.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstddef>

#include "mla_decode.h"
#include "mla_internal.h"
#include "mla_ptx.cuh"
#include "mla_schedule.cuh"
#include "mla_window.cuh"

namespace mla {

constexpr int kRowsPerCta = 64;           // query rows per CTA = MMA N
constexpr int kChunks = 9;                // 576 / 64 columns
constexpr int kChunkBytes = kTileTokens * 64 * 2;   // 16 KB
constexpr int kQChunkBytes = kRowsPerCta * 64 * 2;  // 8 KB
constexpr int kSmemKv = 0;
constexpr int kSmemQ = kChunks * kChunkBytes;                 // 147456
constexpr int kSmemSmall = kSmemQ + kChunks * kQChunkBytes;   // 221184
constexpr int kNumBarriers = 3 * kChunks + 4;
constexpr int kSmallBytes = 8 * kNumBarriers + 16 + 5 * 4 * 4 * 4 * 16;
constexpr int kSmemBytes = kSmallBytes + kSmemSmall + 1024;   // + alignment slack
constexpr int kSmemWork = (kSmemSmall + kSmallBytes + 15) / 16 * 16;  // windowed: the list of pieces
constexpr int kSmemBytesWindow = kSmemWork + 2688 + 1024;
static_assert(kSmemBytesWindow <= 232448, "dynamic shared memory per CTA");
constexpr int kSoftmaxGroups = 4;                  // warpgroups on the softmax
constexpr int kRowsPerGroup = kRowsPerCta / kSoftmaxGroups;  // 16 query rows each
constexpr int kSoftmaxWarp0 = 0;
constexpr int kProducerWarp = 4 * kSoftmaxGroups;
constexpr int kMmaWarp = kProducerWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 1);
// A later tile moves the softmax reference only when a score exceeds it by
// more than this (log2 units): probabilities stay <= 2^8, exact in range.
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;     // O^T: 4 blocks of 64 columns
constexpr uint32_t kTmemS = 256;   // S^T: 64 columns
constexpr uint32_t kIdescQK = idesc_bf16(128, kRowsPerCta, false, false);
constexpr uint32_t kIdescPV = idesc_bf16(128, kRowsPerCta, true, true);

enum class KvMode : int { kPagedBf16 = 0, kSparseBf16 = 1, kPagedFp8 = 2, kPagedFp8V41 = 3 };

// kPagedFp8: the 656-byte cache (fp32 scale per 128 latent codes, bf16 RoPE
// chunk); kPagedFp8V41: the 528-byte cache (FlashMLA README, "FP8 / FP4 KV
// Cache Format", V4.1): 512 e4m3 codes covering all 512 dimensions and 16
// e8m0 scales (one per 32 codes) at byte 512 of the token.  Keys and values
// are then 512 wide: QK^T runs over 8 chunks (no RoPE chunk) and P.V over
// the same 8 chunks.
__host__ __device__ constexpr bool is_fp8(KvMode m) {
  return m == KvMode::kPagedFp8 || m == KvMode::kPagedFp8V41;
}
__host__ __device__ constexpr int qk_chunks(KvMode m) { return m == KvMode::kPagedFp8V41 ? 8 : 9; }

// FP8 cache token: 512 e4m3 codes, 4 fp32 scales (one per 128 latent
// channels), 64 bf16 RoPE values (FlashMLA "Hopper FP8 sparse decode" note,
// "The FP8 KVCache Format").
constexpr int kFp8TokenBytes = 656;
constexpr int kFp8ScaleOffset = 512;
constexpr int kFp8RopeOffset = 528;
// V4.1 cache token (FlashMLA README, "FP8 / FP4 KV Cache Format"): 512 e4m3
// codes, then 16 e8m0 scales (one per 32 codes) at byte 512.
constexpr int kFp8V41TokenBytes = 528;
constexpr int kV41HeadDim = 512;
constexpr uint32_t kDequantBarrier = 5;  // FP8: all softmax warps (1..4: one softmax group each)
// staging of a latent chunk's raw FP8 data inside its own 16 KB bf16 slot
constexpr int kRawScaleOff = 4096;                  // [128 tokens][4 fp32 scales]
constexpr int kRawScaleBytes = kTileTokens * 16;
constexpr int kRawCodeOff = 8192;                   // [128 tokens][64 e4m3 codes]
constexpr int kRawCodeBytes = kTileTokens * 64;
static_assert(kRawScaleOff + kRawScaleBytes <= kRawCodeOff && kRawCodeOff + kRawCodeBytes <= kChunkBytes,
              "staging fits in the slot");

struct SplitParams {
  const int32_t* meta;     // schedule metadata (read-only)
  int32_t* ws_ctrl;        // workspace control words: [0] = the schedule walked (for the combine)
  const int32_t* block_table;
  int64_t bt_stride;       // dense: int32 entries from one block-table row to the next
  int64_t bt_width;        // dense: entries of a row (page slots of a request)
  int64_t num_pages;       // dense: pages in the cache
  const int32_t* cache_seqlens;  // dense: [batch] lengths, checked against the metadata's key counts
  const int32_t* indices;  // sparse: [n_seq, topk]
  const float* attn_sink;  // sparse, optional: [h] sink logits (out scaled by e^lse / (e^lse + e^sink))
  int topk;
  int64_t s_kv;            // sparse: pool rows
  const __nv_bfloat16* kv_rows;  // dense: cache base (L2 prefetch); sparse: pool base
  const __nv_bfloat16* q;        // query rows, for L2 prefetch of the next piece
  const uint8_t* kv_fp8;         // FP8 cache base ([pages, 64, 656] bytes)
  float* ws_o;
  float* ws_lse;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* err;
  int h;
  int d_qk;                // query / key width: 576, or 512 for the V4.1 cache
  int s_q;
  int batch;
  int causal;              // dense: causal flag of the call (checked against the metadata)
  int num_parts;
  int n_hblk;
  int rows;                // query rows loaded per CTA (min(h, 64))
  float scale_log2;        // softmax_scale * log2(e)
  // windowed attention (no metadata): see mla_window.cuh
  const int32_t* new_lens; // optional [batch]
  int window, sinks;
  WindowPlan plan;
};

// The pieces that part `part` walks: next() moves to a piece (tiles [t0, t1) of
// query token q, split `split`); page(e) is the logical page of tile list
// entry e (tile t holds entries 2t, 2t + 1), whole() whether the token's tiles
// are all in this piece, split_row() the piece's row of the split workspace.
// By the schedule metadata:
template <bool kWindow>
struct Pieces {
  const SplitParams& p;
  const int32_t* meta;
  PartCursor cur;
  int q, t0, t1, split;
  __device__ __forceinline__ Pieces(const SplitParams& prm, const int32_t* walked, int part)
      : p(prm), meta(walked), cur(walked_part_cursor(prm.meta, walked, part)) {}
  __device__ __forceinline__ bool next() { return next_piece(meta, p.num_parts, &cur, &q, &t0, &t1, &split); }
  __device__ __forceinline__ const int32_t* rec() const { return meta_seq(meta, p.num_parts, q); }
  __device__ __forceinline__ int32_t keys() const { return rec()[kSKeys]; }
  __device__ __forceinline__ int32_t page(int32_t e) const { return e; }
  __device__ __forceinline__ bool edge(int) const { return false; }
  __device__ __forceinline__ void tile_masks(int, uint32_t (&)[4]) const {}
  __device__ __forceinline__ bool whole() const { return rec()[kSNSplits] == 1; }
  __device__ __forceinline__ int64_t split_row() const { return static_cast<int64_t>(rec()[kSSplitOff] + split); }
  __device__ __forceinline__ int rows() const { return p.h; }              // query rows of q
  __device__ __forceinline__ int peek_rows(int, int block) const { return block; }
  __device__ __forceinline__ int peek_q() const {                         // the next piece's sequence, -1: none
    PartCursor nc = cur;
    int nq, nt0, nt1, ns;
    return next_piece(meta, p.num_parts, &nc, &nq, &nt0, &nt1, &ns) ? nq : -1;
  }
};

// Windowed: what a part walks, worked out 32 items at a time (lane i of one warp,
// item i) into shared memory, from which every role reads it.  With the
// arithmetic in every role the cold start of a short call was bound by fetching
// seven copies of it.
struct WorkItem {
  int32_t q, rows;                                // first query token (of all requests' slots in turn), query rows
  int32_t t0, t1;                                 // tiles of the piece
  int32_t row;                                    // block of the split workspace, -1 for an item that is not cut
  int32_t b, j0;                                  // request, slot of the first token
  int32_t least, most, first, count;              // WindowEnds
  int32_t head_pages, skip;                       // page list
  int32_t edge_head, edge_lo, edge_hi, edge_end;  // tiles with keys not seen
  int32_t pad[3];
};
constexpr int kWorkItems = 32;
struct WorkList {
  WorkItem item[kWorkItems];
  uint64_t full, free;  // a batch is written (one arrival) / every role but the planner's is done with it
  int64_t m;            // the next batch's first item number on the part's cost line
  int32_t line, pl;     // the line, and the part's number on it
  int32_t n, more;      // pieces of the batch; whether another may follow
  uint32_t batches;     // written so far
};
constexpr int kWorkBytes = 2688;
static_assert(sizeof(WorkItem) == 80 && sizeof(WorkList) <= kWorkBytes && kWorkBytes % 128 == 0, "work list");

// Called by a whole warp: the part's next batch of items.  Pieces go into the
// list; tokens that see no key have none: their rows (row0 .. row0 + most - 1 of
// the item's) are zeroed here by the part that owns the item.  Without `commit`
// it goes the same way with a length of its own making, reads nothing that the
// preceding kernel may still be writing, and leaves nothing that counts.
__device__ __noinline__ static void plan_batch(const SplitParams& p, WorkList* list, bool commit, int row0, int most) {
  const WindowPlan& w = p.plan;
  const int lane = threadIdx.x & 31, line = list->line, pl = list->pl;
  const int64_t mine = list->m + lane, item = line + w.lanes * mine;
  const bool in = item < w.items && (w.whole || mine * (w.tiles + w.fixed) < (pl + 1) * w.per);
  WorkItem x = {};
  WindowPiece piece = {};
  if (in) {
    x.b = static_cast<int32_t>(item) / w.chunks;
    x.j0 = (static_cast<int32_t>(item) - x.b * w.chunks) * w.group;
    x.q = x.b * p.s_q + x.j0;
    x.rows = min(w.group, p.s_q - x.j0) * p.h;
    const RequestLengths len = request_lengths(p.cache_seqlens, p.new_lens, p.s_q, x.b, commit);
    const WindowEnds e = item_ends(len.L, len.n, p.s_q, x.j0, w.group);
    const WindowSpan span = window_span(e, p.window, p.sinks);
    piece = window_piece(w, mine, pl, span.tiles);
    x.row = piece.cut ? window_row(w, mine, pl, line) : -1;
    x.t0 = piece.t0; x.t1 = piece.t1;
    x.least = e.least; x.most = e.most; x.first = e.first; x.count = e.count;
    x.head_pages = span.head_pages; x.skip = span.skip;
    x.edge_head = span.edge_head; x.edge_lo = span.edge_lo; x.edge_hi = span.edge_hi; x.edge_end = span.edge_end;
  }
  const uint32_t has = __ballot_sync(0xffffffffu, x.t0 < x.t1);
  if (x.t0 < x.t1) list->item[__popc(has & ((1u << lane) - 1u))] = x;
  const bool more = __all_sync(0xffffffffu, in);
  __syncwarp();
  if (lane == 0) {
    list->n = __popc(has);
    list->more = more ? 1 : 0;
    if (commit) {
      list->m = mine + kWorkItems;
      ++list->batches;
      mbar_arrive(smem_u32(&list->full));
    }
  }
  __syncwarp();
  uint32_t none = commit && most > 0 ? __ballot_sync(0xffffffffu, in && x.most == 0 && piece.owner) : 0u;
  for (; none; none &= none - 1) {
    const int from = __ffs(none) - 1;
    const int q = __shfl_sync(0xffffffffu, x.q, from), rows = min(__shfl_sync(0xffffffffu, x.rows, from) - row0, most);
    const int b = q / p.s_q, j0 = q - b * p.s_q;
    uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(q) * p.h + row0) * kDv);
    for (int i = lane; i < rows * kDv / 8; i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int r = row0 + lane; r < row0 + rows; r += 32)
      p.lse[(static_cast<int64_t>(b) * p.h + r % p.h) * p.s_q + j0 + r / p.h] = -INFINITY;
  }
}

// Called by the planning warp in place of pdl_wait_primary(): the first batch.
// The lengths are only final once the preceding kernel is done, so they are not
// read before the wait; but the way there is gone twice, once before it with a
// made-up length: that fetches the code.  The first item's query rows, length
// and page slots start towards L2 (a prefetch reads nothing).
__device__ __forceinline__ void plan_first(const SplitParams& p, WorkList* list, int part, int row0, int most) {
  const int lane = threadIdx.x & 31;
  const WindowPlan& w = p.plan;
  const int line = part % w.lanes, pl = part / w.lanes;
  const int64_t m = window_first_item(w, pl);
  if (lane == 0) {
    list->line = line; list->pl = pl; list->m = m; list->batches = 0;
  }
  __syncwarp();
  plan_batch(p, list, false, row0, most);
  const int64_t item = line + w.lanes * m;
  if (item < w.items) {
    const int64_t b = item / w.chunks, j0 = (item - b * w.chunks) * w.group;
    const int rows = min(w.group, p.s_q - static_cast<int>(j0)) * p.h;
    if (lane == 0) prefetch_l2(p.q + (b * p.s_q + j0) * p.h * p.d_qk, rows * p.d_qk * 2);
    if (lane == 1) prefetch_line_l2(p.cache_seqlens + b);
    if (lane == 2 && p.new_lens) prefetch_line_l2(p.new_lens + b);
    for (int64_t i = 32 * lane; i < p.bt_width && i < 4096; i += 1024) prefetch_line_l2(p.block_table + b * p.bt_stride + i);
  }
  __syncwarp();
  pdl_wait_primary();
  plan_batch(p, list, true, row0, most);
}

// The roles' side.
template <>
struct Pieces<true> {
  const SplitParams& p;
  uint32_t list;   // shared memory address of the WorkList
  bool warps;      // a role of whole warps (one arrival each), not of one thread
  bool plans;      // the planning warp's role, and the query rows that it writes for items without a key:
  int row0, most;
  int i = 0, n = 0;
  uint32_t batch = 0;
  int q, t0, t1;
  __device__ __forceinline__ Pieces(const SplitParams& prm, WorkList* l, bool whole_warps)
      : p(prm), list(smem_u32(l)), warps(whole_warps), plans(false), row0(0), most(0) {}
  __device__ __forceinline__ void plan_by(bool planner, int first_row, int rows) {
    plans = planner; row0 = first_row; most = rows;
  }
  __device__ __forceinline__ bool next() {
    const uint32_t full = list + offsetof(WorkList, full), free = list + offsetof(WorkList, free);
    while (i == n) {
      // (Every role comes here for every batch, if need be by walk_list_out(), so these end.)
      if (batch > 0) {
        if (ld_shared_i32(list + offsetof(WorkList, more)) == 0) return false;
        if (warps) __syncwarp();
        if (plans) {
          (void)mbar_wait_all_roles(free, (batch - 1) & 1, p.err);
          plan_batch(p, reinterpret_cast<WorkList*>(__cvta_shared_to_generic(list)), true, row0, most);
        } else if (!warps || (threadIdx.x & 31) == 0) {
          mbar_arrive(free);
        }
      }
      if (!mbar_wait_all_roles(full, batch & 1, p.err)) return false;
      ++batch;
      i = 0;
      n = ld_shared_i32(list + offsetof(WorkList, n));
    }
    ++i;
    q = at(offsetof(WorkItem, q)); t0 = at(offsetof(WorkItem, t0)); t1 = at(offsetof(WorkItem, t1));
    return true;
  }
  __device__ __forceinline__ int32_t at(int field) const {  // of the present item
    return ld_shared_i32(list + (i - 1) * static_cast<int>(sizeof(WorkItem)) + field);
  }
  // Query token of the piece after this one, -1 when it is not known.
  __device__ __forceinline__ int peek_q() const { return i < n ? at(sizeof(WorkItem) + offsetof(WorkItem, q)) : -1; }
  __device__ __forceinline__ int peek_rows(int row, int block) const {
    return min(at(sizeof(WorkItem) + offsetof(WorkItem, rows)) - row, block);
  }
  // The end of the token of query row r of the item (0: padding, or a row past
  // the item's tokens).
  __device__ __forceinline__ int32_t end_of_row(int r) const {
    if (r >= rows()) return 0;
    const int j = p.plan.group == 1 ? 0 : r / p.h;
    return item_end(at(offsetof(WorkItem, first)), at(offsetof(WorkItem, count)), j);
  }
  __device__ __forceinline__ int32_t page(int32_t e) const {
    return e < at(offsetof(WorkItem, head_pages)) ? e : e + at(offsetof(WorkItem, skip));
  }
  // position of key k of tile t
  __device__ __forceinline__ int32_t key_at(int t, int k) const { return kPage * page(2 * t + (k >> 6)) + (k & 63); }
  // Whether tile t may hold a key that one of the item's tokens does not see.
  __device__ __forceinline__ bool edge(int t) const {
    return t == at(offsetof(WorkItem, edge_head)) || t >= at(offsetof(WorkItem, edge_end)) ||
           (t >= at(offsetof(WorkItem, edge_lo)) && t <= at(offsetof(WorkItem, edge_hi)));
  }
  // Bit k % 32 of word k / 32: some token of the item sees key k of tile t.
  __device__ __forceinline__ void tile_masks(int t, uint32_t (&seen)[4]) const {
    const int32_t most = keys(), lo = window_lo(at(offsetof(WorkItem, least)), p.window);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t x = kPage * page(2 * t + h);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        seen[2 * h + k] = low_bits(most - x - 32 * k) & (low_bits(p.sinks - x - 32 * k) | ~low_bits(lo - x - 32 * k));
    }
  }
  // Whether any of the item's tokens sees the key at position x.
  __device__ __forceinline__ bool any_sees(int32_t x) const {
    return x < keys() && (x < p.sinks || x >= window_lo(at(offsetof(WorkItem, least)), p.window));
  }
  // Whether some of them see it and others do not (no key, of a single token).
  __device__ __forceinline__ bool some_see(int32_t x) const {
    const int32_t all_lo = window_lo(keys(), p.window);
    return any_sees(x) && !(x < at(offsetof(WorkItem, least)) && (x < p.sinks || x >= all_lo));
  }
  __device__ __forceinline__ int rows() const { return at(offsetof(WorkItem, rows)); }  // of its request's token slots
  __device__ __forceinline__ int b() const { return at(offsetof(WorkItem, b)); }
  __device__ __forceinline__ int j0() const { return at(offsetof(WorkItem, j0)); }
  __device__ __forceinline__ int32_t keys() const { return at(offsetof(WorkItem, most)); }
  __device__ __forceinline__ bool whole() const { return at(offsetof(WorkItem, row)) < 0; }
  __device__ __forceinline__ int64_t split_row() const { return at(offsetof(WorkItem, row)); }
};

template <bool kWindow>
__device__ __forceinline__ Pieces<kWindow> role_pieces(const SplitParams& p, const int32_t* meta, int part,
                                                       WorkList* work, bool whole_warps) {
  if constexpr (kWindow) return Pieces<true>(p, work, whole_warps);
  else return Pieces<false>(p, meta, part);
}

struct SmemSmall {
  // float arrays first: each row of 32 floats is read back as float4 vectors,
  // so every row must start on a 16-byte boundary.
  alignas(16) float red_max[kSoftmaxGroups][4][kRowsPerGroup];
  alignas(16) float red_sum[kSoftmaxGroups][4][kRowsPerGroup];
  alignas(16) float red_bsum[kSoftmaxGroups][4][kRowsPerGroup];
  alignas(16) float bcast[kSoftmaxGroups][4][kRowsPerGroup];
  alignas(16) float bcast2[kSoftmaxGroups][4][kRowsPerGroup];
  uint64_t full[kChunks];
  uint64_t empty[kChunks];
  uint64_t raw_full[kChunks - 1];  // FP8: raw codes and scales of a latent chunk landed
  uint64_t q_full, q_empty, s_full, p_full, o_done;
  uint32_t tmem_base;
  uint32_t abort;
};
static_assert(offsetof(SmemSmall, bcast) % 16 == 0 && offsetof(SmemSmall, bcast2) % 16 == 0,
              "broadcast rows are read as float4");
static_assert(offsetof(SmemSmall, full) % 8 == 0, "mbarriers are 8-byte objects");
static_assert(sizeof(SmemSmall) <= kSmallBytes, "small smem region");

// Reduce 32 per-thread values (one per query row of this warpgroup) over the
// warp's 32 lanes, leaving in lane l the reduction for row l.  Recursive
// halving: at each step a lane keeps the half of its vector that its lane bit
// selects and adds the partner's copy of that half.
template <bool kMax>
__device__ __forceinline__ float warp_reduce_scatter32(const float (&v)[32], int lane) {
  float a[16], b[8], c[4], d[2];
  bool hi = lane & 16;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float send = hi ? v[i] : v[i + 16];
    const float keep = hi ? v[i + 16] : v[i];
    const float r = __shfl_xor_sync(0xffffffffu, send, 16);
    a[i] = kMax ? fmaxf(keep, r) : keep + r;
  }
  hi = lane & 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float send = hi ? a[i] : a[i + 8];
    const float keep = hi ? a[i + 8] : a[i];
    const float r = __shfl_xor_sync(0xffffffffu, send, 8);
    b[i] = kMax ? fmaxf(keep, r) : keep + r;
  }
  hi = lane & 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float send = hi ? b[i] : b[i + 4];
    const float keep = hi ? b[i + 4] : b[i];
    const float r = __shfl_xor_sync(0xffffffffu, send, 4);
    c[i] = kMax ? fmaxf(keep, r) : keep + r;
  }
  hi = lane & 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float send = hi ? c[i] : c[i + 2];
    const float keep = hi ? c[i + 2] : c[i];
    const float r = __shfl_xor_sync(0xffffffffu, send, 2);
    d[i] = kMax ? fmaxf(keep, r) : keep + r;
  }
  hi = lane & 1;
  const float send = hi ? d[0] : d[1];
  const float keep = hi ? d[1] : d[0];
  const float r = __shfl_xor_sync(0xffffffffu, send, 1);
  return kMax ? fmaxf(keep, r) : keep + r;
}

// Sum of 16 per-thread values (one per query row of the warpgroup) over the
// warp's 32 lanes; lanes l and l + 16 both end with the sum for row l & 15.
__device__ __forceinline__ float warp_sum_scatter16(const float (&v)[16], int lane) {
  float a[16], b[8], c[4], d[2];
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = v[i] + __shfl_xor_sync(0xffffffffu, v[i], 16);
  bool hi = lane & 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float send = hi ? a[i] : a[i + 8];
    const float keep = hi ? a[i + 8] : a[i];
    b[i] = keep + __shfl_xor_sync(0xffffffffu, send, 8);
  }
  hi = lane & 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float send = hi ? b[i] : b[i + 4];
    const float keep = hi ? b[i + 4] : b[i];
    c[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
  }
  hi = lane & 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float send = hi ? c[i] : c[i + 2];
    const float keep = hi ? c[i + 2] : c[i];
    d[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
  }
  hi = lane & 1;
  const float send = hi ? d[0] : d[1];
  const float keep = hi ? d[1] : d[0];
  return keep + __shfl_xor_sync(0xffffffffu, send, 1);
}

__device__ __forceinline__ void load_bcast32(const float* src, float (&dst)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 t = *reinterpret_cast<const float4*>(src + i);
    dst[i] = t.x; dst[i + 1] = t.y; dst[i + 2] = t.z; dst[i + 3] = t.w;
  }
}

// Physical page of logical page `pg` of a sequence with `keys` keys whose
// block-table row is `bt_row`, or -1 when there is none: the entry is outside
// [0, num_pages), or the page slot lies past the row's bt_width entries
// (more keys than the row can address).  Pages past the last one of the
// sequence (the second page of a tile's last 64-key half) map to the last.
__device__ __forceinline__ int32_t page_of(const SplitParams& p, const int32_t* bt_row, int32_t keys,
                                           int pg) {
  const int last = (keys - 1) / kPage;
  const int slot = pg < last ? pg : last;
  if (static_cast<int64_t>(slot) >= p.bt_width) return -1;
  const int32_t blk = bt_row[slot];
  return (blk < 0 || static_cast<int64_t>(blk) >= p.num_pages) ? -1 : blk;
}

// Block-table row of sequence q (request q / s_q).
__device__ __forceinline__ const int32_t* bt_row_of(const SplitParams& p, int q) {
  return p.block_table + static_cast<int64_t>(q / p.s_q) * p.bt_stride;
}

// Dense: flags MLA_DEVERR_METADATA when the metadata's key count for sequence
// q differs from the one cache_seqlens and the causal flag give (metadata
// computed from other lengths).  The kernels keep walking the metadata's
// tiles; page_of keeps every block-table read inside its row.
__device__ __forceinline__ void check_seq_keys(const SplitParams& p, int q, int32_t keys) {
  if (!p.cache_seqlens) return;
  const int32_t want = seq_keys(p.cache_seqlens, q / p.s_q, q % p.s_q, p.s_q, p.causal, 0);
  if (want != keys && p.err) atomicOr(p.err, MLA_DEVERR_METADATA);
}

// Sparse: the first index among a query's n_slots index slots that names a
// pool row (warp-wide; every lane gets it), or 0 when there is none.
// Invalid slots are loaded from a row the query does name, so a masked slot
// (weight 0) never multiplies a row the caller did not ask for: 0 * NaN is
// NaN, and rows the query does not name may hold anything.
__device__ __forceinline__ int32_t first_valid_index(const int32_t* idx_row, int n_slots, int64_t s_kv,
                                                     int lane) {
  for (int base = 0; base < n_slots; base += 32) {
    const int slot = base + lane;
    const int32_t id = slot < n_slots ? idx_row[slot] : -1;
    const uint32_t m = __ballot_sync(0xffffffffu, id >= 0 && static_cast<int64_t>(id) < s_kv);
    if (m) return __shfl_sync(0xffffffffu, id, __ffs(m) - 1);
  }
  return 0;
}

// Sparse: the pool rows a warp loads for one 128-slot tile, lane L owning
// slots 4L .. 4L + 3 (id: the index list entries, -1 past the key count).
// Slots that name no row (-1, out of range) take the first row named in the
// tile, or, in a tile with none, the first row the query names (found by a
// scan of its list, `fallback`, computed once and cached in *fallback_cache,
// -2 = not yet known).  Out-of-range entries other than -1 set
// MLA_DEVERR_BAD_INDEX (when `flag`).
__device__ __forceinline__ void sparse_rows4(const SplitParams& p, const int32_t (&id)[4], int lane,
                                             const int32_t* idx_row, int n_slots, bool flag,
                                             int32_t* fallback_cache, int32_t (&y)[4]) {
  bool valid[4];
  int32_t first = -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    valid[i] = id[i] >= 0 && static_cast<int64_t>(id[i]) < p.s_kv;
    if (!valid[i] && id[i] != -1 && flag && p.err) atomicOr(p.err, MLA_DEVERR_BAD_INDEX);
    if (valid[i] && first < 0) first = id[i];
  }
  const uint32_t any = __ballot_sync(0xffffffffu, first >= 0);
  int32_t sub;
  if (any) {
    sub = __shfl_sync(0xffffffffu, first, __ffs(any) - 1);
  } else {
    if (*fallback_cache == -2) *fallback_cache = first_valid_index(idx_row, n_slots, p.s_kv, lane);
    sub = *fallback_cache;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = valid[i] ? id[i] : sub;
}

// FP8 cache: 16 e4m3 codes of token dq_r (unit dq_u of a 64-code chunk) times
// their fp32 scale, rounded to bf16, into the chunk's 128-byte-swizzled row
// `row` (shared memory).  Kept out of line: inlined into the softmax loop it
// pushed that loop past the 96 registers a thread of this kernel may hold.
static __device__ __noinline__ void convert_unit(uint32_t row, int dq_r, int dq_u, uint4 codes, float sc) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t w0 = half ? codes.z : codes.x, w1 = half ? codes.w : codes.y;
    const float2 a0 = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w0 & 0xFFFFu)));
    const float2 a1 = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w0 >> 16)));
    const float2 a2 = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w1 & 0xFFFFu)));
    const float2 a3 = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w1 >> 16)));
    st_shared_v4(row + ((2 * dq_u + half) ^ (dq_r & 7)) * 16, pack_bf16x2(a0.x * sc, a0.y * sc),
                 pack_bf16x2(a1.x * sc, a1.y * sc), pack_bf16x2(a2.x * sc, a2.y * sc),
                 pack_bf16x2(a3.x * sc, a3.y * sc));
  }
}

extern __shared__ uint8_t smem_raw[];
__device__ __forceinline__ uint8_t* smem_aligned() {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
}

// Windowed: a role that has left its loop over the pieces after a failed wait goes
// on through the work list, whose batches need every role's arrival.  (The batch
// that it was in is the last one written, since the next waits for it; a role that
// has walked them all finds no more.)  All is worked out here, so that the loops
// keep their registers.
__device__ __noinline__ static void walk_list_out(const SplitParams& p) {
  const int warp = threadIdx.x >> 5;
  WorkList* list = reinterpret_cast<WorkList*>(smem_aligned() + kSmemWork);
  Pieces<true> pc(p, list, warp < kProducerWarp);
  pc.plan_by(warp == kSoftmaxWarp0, static_cast<int>(blockIdx.x) % p.n_hblk * kRowsPerCta, kRowsPerCta);
  pc.batch = ld_shared_i32(smem_u32(&list->batches));
  while (pc.next()) pc.i = pc.n;
}

// Windowed: what is not finite in two chunks of some of 32 keys becomes zero (`keys`:
// a bit each; row0: the first key's row of the first chunk).  Called by a whole
// warp: half of it takes the 16 units of a key, two keys at a time (a thread per
// key: 16 heads of two tokens over 512 keys 27.2 -> 29.8 us).
__device__ __noinline__ static void finite_keys(uint32_t keys, uint32_t row0) {
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t unit = row0 + ((lane >> 3) & 1) * kChunkBytes + (lane & 7) * 16;
  while (keys) {
    const int first = __ffs(keys) - 1;
    keys &= keys - 1;
    const int second = keys ? __ffs(keys) - 1 : first;
    keys &= keys - 1;
    finite_unit(unit + (lane < 16 ? first : second) * 128);
  }
}

template <KvMode kMode, bool kWindow = false>
__global__ void __launch_bounds__(kThreads, 1)
    mla_splitkv_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_kv,
                       const __grid_constant__ CUtensorMap tm_codes,
                       const __grid_constant__ CUtensorMap tm_scales,
                       const __grid_constant__ SplitParams p) {
  uint8_t* smem = smem_aligned();
  SmemSmall* sm = reinterpret_cast<SmemSmall*>(smem + kSmemSmall);
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t kv_base = smem_base + kSmemKv;
  const uint32_t q_base = smem_base + kSmemQ;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x / p.n_hblk;
  const int hb = blockIdx.x % p.n_hblk;
  [[maybe_unused]] WorkList* work = reinterpret_cast<WorkList*>(smem + kSmemWork);  // windowed
  // The metadata must describe this call; otherwise nothing is read or written.
  // (A windowed call has no metadata.)
  const bool meta_ok = kWindow || meta_header_matches(p.meta, p.batch, p.s_q, p.num_parts, p.topk, p.causal);
  // Schedule B (whole sequences) only when nearly balanced: a tile of this
  // kernel takes ~3-6 us, so the ~26 us that splitting costs is ~4 tiles.
  constexpr int kSplitPenalty = 4;
  const int32_t* meta = !kWindow && meta_ok ? schedule_for(p.meta, kSplitPenalty) : p.meta;
  if (!kWindow && blockIdx.x == 0 && threadIdx.x == 32 * kSoftmaxWarp0) {  // a softmax thread: nothing to do yet
    // read by the combine after this grid: the schedule walked, or -1 when
    // the metadata was rejected (the combine then writes nothing), and
    // whether that schedule left anything to merge or fill
    p.ws_ctrl[1] = (meta_ok && (meta == p.meta || meta[kHTotalSplits] != meta[kHNSeq])) ? 1 : 0;
    p.ws_ctrl[0] = meta_ok ? (meta == p.meta ? 0 : 1) : -1;
    if (!meta_ok && p.err) atomicOr(p.err, MLA_DEVERR_METADATA);
  }

  // ---- setup: barriers, TMEM, zeroed padding rows of Q
  // FP8 with two head blocks: each CTA converts half of the latent chunks
  // (chunk c by head block c mod 2) and copies them into the peer's slots
  const bool share = is_fp8(kMode) && p.n_hblk == 2;
  constexpr int kQk = qk_chunks(kMode);  // key chunks of QK^T
  if (threadIdx.x == 0) {
    for (int c = 0; c < kChunks; ++c) {
      // FP8: a latent chunk is filled by this CTA's softmax warps (one
      // arrive each), or by one bulk copy from the peer (one local arm + bytes)
      const bool from_peer = share && c < kChunks - 1 && (c & 1) != hb;
      mbar_init(smem_u32(&sm->full[c]),
                (is_fp8(kMode) && c < kChunks - 1 && !from_peer) ? 4 * kSoftmaxGroups : 1);
      // a slot is free once the MMA threads of every CTA writing into it
      // have released it
      mbar_init(smem_u32(&sm->empty[c]), (share && c < kChunks - 1) ? 2 : 1);
    }
    for (int c = 0; c < kChunks - 1; ++c) mbar_init(smem_u32(&sm->raw_full[c]), 1);
    mbar_init(smem_u32(&sm->q_full), 1);
    mbar_init(smem_u32(&sm->q_empty), 1);
    mbar_init(smem_u32(&sm->s_full), 1);
    mbar_init(smem_u32(&sm->p_full), 4 * kSoftmaxGroups);  // one arrive per softmax warp
    mbar_init(smem_u32(&sm->o_done), 1);
    if constexpr (kWindow) {
      mbar_init(smem_u32(&work->full), 1);
      mbar_init(smem_u32(&work->free), 4 * kSoftmaxGroups + 1);  // all roles but the planning softmax warp
    }
    sm->abort = 0;
    fence_mbarrier_init();
    // the first tile's arm of every chunk the peer converts (the MMA thread
    // re-arms after each use)
    if (share)
      for (int c = hb ^ 1; c < kChunks - 1; c += 2) mbar_arrive_expect_tx(smem_u32(&sm->full[c]), kChunkBytes);
  }
  if (p.rows < kRowsPerCta) {
    // Rows [rows, 64) of every Q chunk are never written by TMA; zero them
    // once so the padded columns of S^T stay finite.
    const int pad_units = (kRowsPerCta - p.rows) * 8;
    for (int i = threadIdx.x; i < kChunks * pad_units; i += kThreads) {
      const int c = i / pad_units, k = i % pad_units;
      st_shared_v4(q_base + c * kQChunkBytes + p.rows * 128 + k * 16, 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sm->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kv);
    if (is_fp8(kMode)) {
      tma_prefetch_desc(&tm_codes);
      tma_prefetch_desc(&tm_scales);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (share) cluster_sync();  // peers' barriers are initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  volatile uint32_t* abort_flag = &sm->abort;

  if constexpr (kWindow) {
    // everything above overlaps the previous kernel of the stream
    if (warp == kSoftmaxWarp0) plan_first(p, work, part, hb * kRowsPerCta, kRowsPerCta);
    else pdl_wait_primary();
    pdl_launch_dependents();  // the merge may launch now; it waits for this grid to finish
  }

  if (!meta_ok) {
    // nothing to do: every role is skipped, the teardown below still runs
  } else if (is_fp8(kMode) && warp == kProducerWarp) {
    // ===================================================== producer (FP8)
    // Lane 0 loads Q, the bf16 RoPE columns (chunk 8; 656-byte cache only) and, for every latent
    // chunk this CTA converts, the raw e4m3 codes and token scales by TMA into
    // that chunk's own slot (codes at +8 KB, scales at +4 KB), each as soon as
    // the slot is released; the softmax warps convert the slot in place.
    // With two head blocks, each converted slot then goes to the peer CTA's
    // slot by one bulk copy (the peer's MMA thread has armed its barrier).
    if (lane == 0) {
      const int own0 = share ? hb : 0, own_step = share ? 2 : 1;
      const int n_own = (kChunks - 1) / own_step;
      const int n_req = kMode == KvMode::kPagedFp8V41 ? n_own : n_own + 1;  // + the RoPE chunk
      auto pc = role_pieces<kWindow>(p, meta, part, work, false);
      uint32_t tile_ctr = 0, item_ctr = 0;
      bool ok = true;
      const uint64_t pol = l2_policy_evict_first();
      while (ok && pc.next()) {
        const int q = pc.q, t0 = pc.t0, t1 = pc.t1;
        ok = mbar_wait(smem_u32(&sm->q_empty), (item_ctr & 1) ^ 1, abort_flag, p.err);
        if (!ok) break;
        mbar_arrive_expect_tx(smem_u32(&sm->q_full), kQk * p.rows * 128);
        const int q_row = q * p.h + hb * kRowsPerCta;
        for (int c = 0; c < kQk; ++c)
          tma_load_2d(q_base + c * kQChunkBytes, &tm_q, c * 64, q_row, smem_u32(&sm->q_full),
                      l2_policy_evict_last());
        const int32_t keys = pc.keys();
        const int32_t* bt_row = bt_row_of(p, q);
        if constexpr (!kWindow) check_seq_keys(p, q, keys);
        for (int t = t0; t < t1 && ok; ++t) {
          const uint32_t par = (tile_ctr & 1) ^ 1;
          int32_t blk[2];
          for (int h2 = 0; h2 < 2; ++h2) {
            blk[h2] = page_of(p, bt_row, keys, pc.page(2 * t + h2));
            if (blk[h2] < 0) {
              if (p.err) atomicOr(p.err, MLA_DEVERR_BAD_PAGE);
              blk[h2] = static_cast<int32_t>(p.num_pages);  // out of range: TMA fills zeros, codes and scales
            }
          }
          // requests 0 .. n_own - 1: raw data of the owned latent chunks;
          // request n_own: the RoPE chunk (its slot also carries P until the
          // previous tile's P.V is done)
          int issued = 0;
          auto slot_of = [&](int i) { return i == n_own ? kChunks - 1 : own0 + own_step * i; };
          auto issue = [&](int i) {
            if (i == n_own) {
              const uint32_t bar = smem_u32(&sm->full[kChunks - 1]);
              mbar_arrive_expect_tx(bar, kChunkBytes);
              const uint32_t dst = kv_base + (kChunks - 1) * kChunkBytes;
              tma_load_2d(dst, &tm_kv, 0, blk[0] * kPage, bar, pol);
              tma_load_2d(dst + kChunkBytes / 2, &tm_kv, 0, blk[1] * kPage, bar, pol);
              return;
            }
            const int c = own0 + own_step * i;
            const uint32_t bar = smem_u32(&sm->raw_full[c]);
            const uint32_t slot = kv_base + c * kChunkBytes;
            mbar_arrive_expect_tx(bar, kRawCodeBytes + kRawScaleBytes);
            for (int h2 = 0; h2 < 2; ++h2) {
              tma_load_2d(slot + kRawCodeOff + h2 * (kRawCodeBytes / 2), &tm_codes, c * 64,
                          blk[h2] * kPage, bar, pol);
              tma_load_2d(slot + kRawScaleOff + h2 * (kRawScaleBytes / 2), &tm_scales, 0,
                          blk[h2] * kPage, bar);
            }
          };
          for (int k = 0; k < n_own && ok; ++k) {
            while (ok && issued <= k) {
              ok = mbar_wait(smem_u32(&sm->empty[slot_of(issued)]), par, abort_flag, p.err);
              if (ok) issue(issued++);
            }
            if (!share || !ok) continue;
            // chunk k converted: copy it to the peer; while waiting, make
            // every later request whose slot has been released
            const int c = own0 + own_step * k;
            const uint32_t fbar = smem_u32(&sm->full[c]);
            const uint64_t t_start = globaltimer_ns();
            while (ok && !mbar_try_wait_hint(fbar, tile_ctr & 1, 200)) {
              while (issued < n_req && mbar_test_wait(smem_u32(&sm->empty[slot_of(issued)]), par))
                issue(issued++);
              if (*abort_flag) {
                ok = false;
              } else if (globaltimer_ns() - t_start > kWaitTimeoutNs) {
                *abort_flag = 1u;
                if (p.err) atomicOr(p.err, MLA_DEVERR_TIMEOUT);
                ok = false;
              }
            }
            if (ok) {
              const uint32_t slot = kv_base + c * kChunkBytes;
              bulk_copy_to_peer(mapa_shared(slot, hb ^ 1), slot, kChunkBytes,
                                mapa_shared(fbar, hb ^ 1));
            }
          }
          if (t + 1 < t1 && (!share || hb == 0)) {
            // the next tile's pages into L2, behind this tile's own requests (150
            // requests of 64 heads over 4000 keys: 233 us, 224 so; before them a
            // piece of three tiles lost 5 %)
            constexpr int kPageBytes = kPage * (kMode == KvMode::kPagedFp8V41 ? kFp8V41TokenBytes : kFp8TokenBytes);
            for (int h2 = 0; h2 < 2; ++h2) {
              const int32_t nb = page_of(p, bt_row, keys, pc.page(2 * t + 2 + h2));
              if (nb >= 0) prefetch_l2(p.kv_fp8 + static_cast<int64_t>(nb) * kPageBytes, kPageBytes);
            }
          }
          while (ok && issued < n_req) {  // the RoPE chunk, if still due
            ok = mbar_wait(smem_u32(&sm->empty[slot_of(issued)]), par, abort_flag, p.err);
            if (ok) issue(issued++);
          }
          ++tile_ctr;
        }
        ++item_ctr;
      }
    }
  } else if (warp == kProducerWarp && kMode == KvMode::kSparseBf16) {
    // ===================================================== producer (gather)
    // Lane L gathers rows 4L..4L+3 of each 128-row tile with one tile::gather4
    // per column chunk; lane 0 owns the barriers.  Invalid slots (-1, out of
    // range, past topk) fetch pool row 0 and are masked by the softmax.
    auto pc = role_pieces<kWindow>(p, meta, part, work, false);
    uint32_t tile_ctr = 0, item_ctr = 0;
    int32_t issued[kChunks];  // tile counter of each slot's latest gather, -1 = none
    for (int c = 0; c < kChunks; ++c) issued[c] = -1;
    bool ok = true;
    while (ok && pc.next()) {
      const int q = pc.q, t0 = pc.t0, t1 = pc.t1;
      if (lane == 0) {
        ok = mbar_wait(smem_u32(&sm->q_empty), (item_ctr & 1) ^ 1, abort_flag, p.err);
        if (ok) {
          mbar_arrive_expect_tx(smem_u32(&sm->q_full), kChunks * p.rows * 128);
          const int q_row = q * p.h + hb * kRowsPerCta;
          for (int c = 0; c < kChunks; ++c)
            tma_load_2d(q_base + c * kQChunkBytes, &tm_q, c * 64, q_row, smem_u32(&sm->q_full),
                        l2_policy_evict_last());
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      const int32_t* idx_row = p.indices + static_cast<int64_t>(q) * p.topk;
      const int32_t n_slots = pc.keys();  // topk or topk_length
      int32_t fallback = -2;  // first row the query names, found when a tile names none
      for (int t = t0; t < t1 && ok; ++t) {
        int32_t id[4], rid[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int slot = t * kTileTokens + 4 * lane + i;
          id[i] = slot < n_slots ? idx_row[slot] : -1;
        }
        sparse_rows4(p, id, lane, idx_row, n_slots, true, &fallback, rid);
        const uint32_t par = (tile_ctr & 1) ^ 1;
        for (int c = 0; c < kChunks; ++c) {
          if (lane == 0) {
            ok = mbar_wait(smem_u32(&sm->empty[c]), par, abort_flag, p.err);
            if (ok) mbar_arrive_expect_tx(smem_u32(&sm->full[c]), kChunkBytes);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          tma_gather4(kv_base + c * kChunkBytes + 4 * lane * 128, &tm_kv, c * 64, rid[0], rid[1],
                      rid[2], rid[3], smem_u32(&sm->full[c]));
          issued[c] = static_cast<int32_t>(tile_ctr);
        }
        ++tile_ctr;
      }
      ++item_ctr;
    }
    if (!ok && lane == 0) {
      // Let gathers already in flight land before the CTA exits.
      for (int c = 0; c < kChunks; ++c) {
        if (issued[c] < 0) continue;
        const uint64_t t_start = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&sm->full[c]), static_cast<uint32_t>(issued[c]) & 1u) &&
               globaltimer_ns() - t_start < 1000000ull) {
        }
      }
    }
  } else if (warp == kProducerWarp) {
    // ===================================================== producer (TMA)
    if (lane == 0) {
      const uint64_t pol_kv = l2_policy_evict_first();
      const uint64_t pol_q = l2_policy_evict_last();
      auto pc = role_pieces<kWindow>(p, meta, part, work, false);
      uint32_t tile_ctr = 0, item_ctr = 0;
      int32_t issued[kChunks];  // tile counter of each slot's latest load, -1 = none
      for (int c = 0; c < kChunks; ++c) issued[c] = -1;
      bool ok = true;
      while (ok && pc.next()) {
        const int q = pc.q, t0 = pc.t0, t1 = pc.t1;
        // Q rows of this block: 9 boxes of [rows x 64 columns]
        ok = mbar_wait(smem_u32(&sm->q_empty), (item_ctr & 1) ^ 1, abort_flag, p.err);
        if (!ok) break;
        mbar_arrive_expect_tx(smem_u32(&sm->q_full), kChunks * p.rows * 128);
        const int q_row = q * p.h + hb * kRowsPerCta;
        for (int c = 0; c < kChunks; ++c)
          tma_load_2d(q_base + c * kQChunkBytes, &tm_q, c * 64, q_row, smem_u32(&sm->q_full), pol_q);
        {  // the next piece's query rows into L2
          const int nq = pc.peek_q();
          if (nq >= 0)
            prefetch_l2(p.q + (static_cast<int64_t>(nq) * p.h + hb * kRowsPerCta) * p.d_qk,
                        pc.peek_rows(hb * kRowsPerCta, p.rows) * p.d_qk * 2);
        }
        const int32_t keys = pc.keys();
        const int32_t* bt_row = bt_row_of(p, q);
        if constexpr (!kWindow) check_seq_keys(p, q, keys);
        for (int t = t0; t < t1 && ok; ++t) {
          int32_t y[2];
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            int32_t blk = page_of(p, bt_row, keys, pc.page(2 * t + h2));
            if (blk < 0) {
              if (p.err) atomicOr(p.err, MLA_DEVERR_BAD_PAGE);
              blk = static_cast<int32_t>(p.num_pages);  // out of range: TMA fills zeros
            }
            y[h2] = blk * kPage;
          }
          const uint32_t par = (tile_ctr & 1) ^ 1;
          for (int c = 0; c < kChunks; ++c) {
            ok = mbar_wait(smem_u32(&sm->empty[c]), par, abort_flag, p.err);
            if (!ok) break;
            const uint32_t bar = smem_u32(&sm->full[c]);
            mbar_arrive_expect_tx(bar, kChunkBytes);
            const uint32_t dst = kv_base + c * kChunkBytes;
            tma_load_2d(dst, &tm_kv, c * 64, y[0], bar, pol_kv);
            tma_load_2d(dst + kChunkBytes / 2, &tm_kv, c * 64, y[1], bar, pol_kv);
            issued[c] = static_cast<int32_t>(tile_ctr);
          }
          ++tile_ctr;
        }
        ++item_ctr;
      }
      if (!ok) {
        // Let copies already in flight land before the CTA exits.
        for (int c = 0; c < kChunks; ++c) {
          if (issued[c] < 0) continue;
          const uint64_t t_start = globaltimer_ns();
          while (!mbar_try_wait(smem_u32(&sm->full[c]), static_cast<uint32_t>(issued[c]) & 1u) &&
                 globaltimer_ns() - t_start < 1000000ull) {
          }
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ===================================================== MMA issuer
    if (lane == 0) {
      auto pc = role_pieces<kWindow>(p, meta, part, work, false);
      uint32_t tile_ctr = 0, item_ctr = 0;
      bool ok = true;
      const uint32_t p_base = kv_base + 8 * kChunkBytes;
      while (ok && pc.next()) {
        const int q = pc.q, t0 = pc.t0, t1 = pc.t1;
        ok = mbar_wait(smem_u32(&sm->q_full), item_ctr & 1, abort_flag, p.err);
        if (!ok) break;
        for (int t = t0; t < t1 && ok; ++t) {
          const uint32_t par = tile_ctr & 1;
          // S^T = K_tile . Q^T: A = tile chunk (K-major), B = Q chunk (K-major)
          // (unrolled as far as registers go, with constant descriptor offsets: bf16, 150
          // requests of 64 heads over 4000 keys 156 us rolled, 149 so; 656-byte cache, 100
          // x 2 tokens of 128 heads 563 and 535, every other chunk being the peer's)
          constexpr int kUnrollQk = is_fp8(kMode) ? 2 : kQk;
#pragma unroll kUnrollQk
          for (int c = 0; c < kQk; ++c) {
            // FP8 chunks converted by the peer complete on its bulk copy
            const bool from_peer = share && c < kChunks - 1 && (c & 1) != hb;
            ok = from_peer ? mbar_wait_cluster(smem_u32(&sm->full[c]), par, abort_flag, p.err)
                           : mbar_wait(smem_u32(&sm->full[c]), par, abort_flag, p.err);
            if (!ok) break;
            // next tile's arm: this phase is complete, so the arrive counts
            // toward the next one, before the peer can start its copy
            if (from_peer) mbar_arrive_expect_tx(smem_u32(&sm->full[c]), kChunkBytes);
            tc_fence_after();
            const uint64_t a = sw128_desc(kv_base + c * kChunkBytes, 16, 1024);
            const uint64_t bq = sw128_desc(q_base + c * kQChunkBytes, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16_ss(tmem + kTmemS, a + static_cast<uint64_t>((32 * k) >> 4), bq + static_cast<uint64_t>((32 * k) >> 4),
                          kIdescQK, (c | k) != 0);
          }
          if (!ok) break;
          if (t == t1 - 1) mma_commit(smem_u32(&sm->q_empty));
          mma_commit(smem_u32(&sm->s_full));
          // O^T += V^T . P^T: A = tile chunks 2m, 2m+1 read MN-major (the 64
          // latent columns of a chunk are contiguous), B = P^T in slot 8
          // (MN-major: the 64 rows of a token are contiguous)
          ok = mbar_wait(smem_u32(&sm->p_full), par, abort_flag, p.err);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = sw128_desc(kv_base, kChunkBytes, 1024), pd = sw128_desc(p_base, kChunkBytes, 1024);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int s = 0; s < 8; ++s)
              mma_bf16_ss(tmem + kTmemO + 64 * m, vd + static_cast<uint64_t>((2 * m * kChunkBytes + 2048 * s) >> 4),
                          pd + static_cast<uint64_t>((2048 * s) >> 4), kIdescPV, (t != t0 || s != 0) ? 1u : 0u);
            if (share) {  // the slot is written by both CTAs' converters
              mma_commit_multicast(smem_u32(&sm->empty[2 * m]), 0x3);
              mma_commit_multicast(smem_u32(&sm->empty[2 * m + 1]), 0x3);
            } else {
              mma_commit(smem_u32(&sm->empty[2 * m]));
              mma_commit(smem_u32(&sm->empty[2 * m + 1]));
            }
          }
          mma_commit(smem_u32(&sm->empty[8]));
          if (t == t1 - 1) mma_commit(smem_u32(&sm->o_done));
          ++tile_ctr;
        }
        ++item_ctr;
      }
    }
  } else if (warp >= kSoftmaxWarp0 && warp < kSoftmaxWarp0 + 4 * kSoftmaxGroups) {
    // ===================================================== softmax / epilogue
    // Thread = one token row r of the tile (TMEM lane) x the 16 query rows of
    // its warpgroup (TMEM columns).  Probabilities are taken against a per-row
    // reference max m (log2 units).  The first tile of a piece sets m to the
    // exact column max.  A later tile keeps m unless one of its scores exceeds
    // the smallest reference by more than kRescaleLog2 (one warp max and one
    // barrier vote decide); then every row's m moves to its exact running max
    // and O^T and the sums are rescaled.  Two running sums per row: of the
    // fp32 probabilities (for the LSE) and of their bf16 roundings, i.e. the
    // weights the PV MMA multiplies (to normalise O), so a stale reference
    // leaves no coherent gain error on the output (flash-attention sparse-MLA
    // article: summing the bf16-rounded p brings the row gain to the noise
    // floor).  Each tile's 16 x 32 per-lane values are reduce-scattered over
    // the warp, so lane l keeps only the running sums of row l & 15 over the
    // warp's tokens; the four warps' sums meet in shared memory at the end.
    constexpr int R = kRowsPerGroup;
    const int g = (warp - kSoftmaxWarp0) >> 2;  // rows R*g .. R*g + R-1
    const int wq = warp & 3;                    // TMEM lane quarter
    const int r = wq * 32 + lane;               // token row of the tile
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_s = tmem + lane_off + kTmemS + R * g;
    const uint32_t t_o = tmem + lane_off + kTmemO + R * g;
    const uint32_t p_slot = kv_base + 8 * kChunkBytes;
    const uint32_t bar_id = 1 + g;
    const int dq_r = (threadIdx.x - 32 * kSoftmaxWarp0) >> 2;  // FP8 conversion: token
    const int dq_u = threadIdx.x & 3;                           // and 16-code unit
    const float NEG_INF = -INFINITY;
    float* red_w = &sm->red_max[g][wq][0];
    float* bc_m = &sm->bcast[g][wq][0];
    float* bc_a = &sm->bcast2[g][wq][0];
    auto pc = role_pieces<kWindow>(p, meta, part, work, true);
    if constexpr (kWindow) pc.plan_by(warp == kSoftmaxWarp0, hb * kRowsPerCta, kRowsPerCta);
    uint32_t tile_ctr = 0, item_ctr = 0;
    bool ok = true;
    while ((!is_fp8(kMode) || ok) && pc.next()) {
      const int q = pc.q, t0 = pc.t0, t1 = pc.t1;
      const int32_t keys = pc.keys();
      const int32_t* idx_row = (kMode == KvMode::kSparseBf16)
                                   ? p.indices + static_cast<int64_t>(q) * p.topk : nullptr;
      float m_true = NEG_INF;  // running max of row R*g + (lane & 15) (-inf: no key yet)
      float m_use = 0.f;       // reference the probabilities are taken against
      float m_low = NEG_INF;   // smallest m_true over the warpgroup's rows
      float lsum = 0.f;        // sum p of row R*g + (lane & 15) over this warp's tokens
      float bsum = 0.f;        // sum bf16(p) of the same row
      for (int t = t0; t < t1; ++t) {
        if constexpr (is_fp8(kMode)) {
          // ---- FP8: convert this tile's owned latent chunks in place.  Thread
          // = (token dq_r, 16-code unit dq_u); reads of the staging finish at
          // the named barrier before any bf16 write lands on it.  Every exit
          // is decided at a barrier, so all 16 warps leave together.
          const int own0 = share ? hb : 0, own_step = share ? 2 : 1;
          [[maybe_unused]] bool seen_dq = true;  // windowed: the same for the key that it converts
          if constexpr (kWindow) seen_dq = pc.any_sees(pc.key_at(t, dq_r));
#pragma unroll 2
          for (int c = own0; c < kChunks - 1; c += own_step) {
            if (lane == 0 && ok) ok = mbar_wait(smem_u32(&sm->raw_full[c]), tile_ctr & 1, abort_flag, p.err);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            const uint32_t slot = kv_base + c * kChunkBytes;
            uint4 codes = ld_shared_v4(slot + kRawCodeOff + dq_r * 64 + dq_u * 16);
            // the unit's scale: fp32 per 128 codes (656-byte cache), or e8m0
            // per 32 codes, 2^(byte - 127) (528-byte cache)
            float sc = kMode == KvMode::kPagedFp8V41
                           ? e8m0_to_f32(ld_shared_u8(slot + kRawScaleOff + dq_r * 16 + 2 * c + (dq_u >> 1)))
                           : ld_shared_f32(slot + kRawScaleOff + dq_r * 16 + (c >> 1) * 4);
            if constexpr (kWindow) {  // keys not seen become zeros: their weight 0 times what is there could be NaN
              if (!seen_dq) {
                codes = make_uint4(0u, 0u, 0u, 0u);
                sc = 0.f;
              }
            }
            ok = !named_barrier_or(kDequantBarrier, 128 * kSoftmaxGroups, !ok);
            if (!ok) break;
            convert_unit(slot + dq_r * 128, dq_r, dq_u, codes, sc);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm->full[c]));
          }
          if (!ok) break;
        }
        // windowed: whether this warpgroup's token, or any of the item's, sees
        // the key of this thread's row
        [[maybe_unused]] bool seen = true, seen_any = true;
        if constexpr (kWindow) {
          const int32_t x = pc.key_at(t, r);
          // (h is a multiple of 16, so the warpgroup's rows are one token's)
          seen = window_sees(pc.end_of_row(hb * kRowsPerCta + R * g), p.window, p.sinks, x);
          seen_any = pc.any_sees(x);
        }
        if (is_fp8(kMode) || ok) ok = mbar_wait(smem_u32(&sm->s_full), tile_ctr & 1, abort_flag, p.err);
        if constexpr (is_fp8(kMode)) {  // leave together (the barrier above)
          ok = !named_barrier_or(kDequantBarrier, 128 * kSoftmaxGroups, !ok);
          if (!ok) break;
        } else {  // a warp whose wait failed goes on to its group's barriers; what it computes no longer counts
          ok = __all_sync(0xffffffffu, ok);
        }
        tc_fence_after();
        float x[R];
        tmem_ld16(t_s, x);
        tmem_wait_ld();
        const int tok = t * kTileTokens + r;
        bool valid = kWindow ? seen : tok < keys;
        if (kMode == KvMode::kSparseBf16 && valid) {
          const int32_t id = idx_row[tok];
          valid = id >= 0 && static_cast<int64_t>(id) < p.s_kv;
        }
        // masked keys: -inf by selection, so a non-finite score of a masked
        // row cannot leak into the max or the sums
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = valid ? x[i] * p.scale_log2 : NEG_INF;
        bool full = true;
        if (t != t0) {
          float u = x[0];
#pragma unroll
          for (int i = 1; i < R; ++i) u = fmaxf(u, x[i]);
          u = warp_max_f32(u);
          full = named_barrier_or(bar_id, 128, u > m_low + kRescaleLog2);
        }
        if (full) {
          // exact column max of this tile over the 128 tokens
#pragma unroll
          for (int i = 0; i < R; i += 4) {
            const float w0 = warp_max_f32(x[i]), w1 = warp_max_f32(x[i + 1]);
            const float w2 = warp_max_f32(x[i + 2]), w3 = warp_max_f32(x[i + 3]);
            if (lane == 0) *reinterpret_cast<float4*>(red_w + i) = make_float4(w0, w1, w2, w3);
          }
          named_barrier_sync(bar_id, 128);
          const int row = lane & (R - 1);
          const float mt = fmaxf(fmaxf(sm->red_max[g][0][row], sm->red_max[g][1][row]),
                                 fmaxf(sm->red_max[g][2][row], sm->red_max[g][3][row]));
          const float m_new = fmaxf(m_true, mt);
          const float m_use_new = (m_new == NEG_INF) ? 0.f : m_new;
          // (windowed: also for a row that has seen no key yet)
          const float alpha = (t == t0 || (kWindow && m_true == NEG_INF)) ? 1.f : fast_exp2(m_use - m_use_new);
          m_true = m_new;
          m_use = m_use_new;
          m_low = warp_min_f32(m_true);
          if (lane < R) {
            bc_m[lane] = m_use;
            bc_a[lane] = alpha;
          }
          __syncwarp();
          if (t != t0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            lsum *= alpha;  // this lane's row is row = lane & 15, whose factor is alpha
            bsum *= alpha;
            // PV of the previous tile completed before s_full of this tile
            // fired (one thread's tcgen05 operations complete in order)
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              float o[R];
              tmem_ld16(t_o + 64 * m, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < R; i += 4) {
                const float4 a4 = *reinterpret_cast<const float4*>(bc_a + i);
                o[i] *= a4.x; o[i + 1] *= a4.y; o[i + 2] *= a4.z; o[i + 3] *= a4.w;
              }
              tmem_st16(t_o + 64 * m, o);
            }
            tmem_wait_st();
          }
        }
        // probabilities against the reference; P^T row r, rows R*g .. R*g+R-1
        // -> 16-byte units 2g, 2g+1 (swizzled)
        const uint32_t prow = p_slot + r * 128;
        float tp[R], tb[R];  // this tile's p and bf16(p) of the lane's token, per row
#pragma unroll
        for (int cu = 0; cu < 2; ++cu) {
          const float4 m0 = *reinterpret_cast<const float4*>(bc_m + 8 * cu);
          const float4 m1 = *reinterpret_cast<const float4*>(bc_m + 8 * cu + 4);
          float e[8];
          e[0] = fast_exp2(x[8 * cu + 0] - m0.x); e[1] = fast_exp2(x[8 * cu + 1] - m0.y);
          e[2] = fast_exp2(x[8 * cu + 2] - m0.z); e[3] = fast_exp2(x[8 * cu + 3] - m0.w);
          e[4] = fast_exp2(x[8 * cu + 4] - m1.x); e[5] = fast_exp2(x[8 * cu + 5] - m1.y);
          e[6] = fast_exp2(x[8 * cu + 6] - m1.z); e[7] = fast_exp2(x[8 * cu + 7] - m1.w);
          uint32_t pk[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            pk[k] = pack_bf16x2(e[2 * k], e[2 * k + 1]);
            tp[8 * cu + 2 * k] = e[2 * k];
            tp[8 * cu + 2 * k + 1] = e[2 * k + 1];
            tb[8 * cu + 2 * k] = __uint_as_float(pk[k] << 16);
            tb[8 * cu + 2 * k + 1] = __uint_as_float(pk[k] & 0xFFFF0000u);
          }
          const uint32_t unit = static_cast<uint32_t>((2 * g + cu) ^ (r & 7));
          st_shared_v4(prow + unit * 16, pk[0], pk[1], pk[2], pk[3]);
        }
        if constexpr (kWindow && !is_fp8(kMode)) {
          // the rows of keys not seen become zeros before P.V reads them (Q.K^T
          // has): their weight 0 times what is there could be NaN
          if (!seen_any) {
            const uint32_t row = kv_base + 2 * g * kChunkBytes + r * 128;
#pragma unroll 1
            for (uint32_t u = lane; u < lane + 8u; ++u) {
              st_shared_v4(row + ((u & 7) << 4), 0u, 0u, 0u, 0u);
              st_shared_v4(row + kChunkBytes + ((u & 7) << 4), 0u, 0u, 0u, 0u);
            }
          }
        }
        if constexpr (kWindow) {
          // a key that other tokens of the item do not see: what is not finite in it
          // becomes zero likewise (a token that does see it is NaN by its score)
          if (p.plan.group > 1) {
            const uint32_t some = __ballot_sync(0xffffffffu, pc.some_see(pc.key_at(t, r)));
            if (some) finite_keys(some, kv_base + 2 * g * kChunkBytes + 32 * wq * 128);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm->p_full));
        lsum += warp_sum_scatter16(tp, lane);  // row lane & 15, this warp's 32 tokens
        bsum += warp_sum_scatter16(tb, lane);
        ++tile_ctr;
      }
      if (is_fp8(kMode) && !ok) break;
      // ---- epilogue: O^T / sum bf16(p) -> out (one split) or fp32 partial
      const int row = lane & (R - 1);
      if (lane < R) {
        sm->red_sum[g][wq][lane] = lsum;
        sm->red_bsum[g][wq][lane] = bsum;
      }
      named_barrier_sync(bar_id, 128);
      lsum = (sm->red_sum[g][0][row] + sm->red_sum[g][1][row]) +
             (sm->red_sum[g][2][row] + sm->red_sum[g][3][row]);
      bsum = (sm->red_bsum[g][0][row] + sm->red_bsum[g][1][row]) +
             (sm->red_bsum[g][2][row] + sm->red_bsum[g][3][row]);
      if (is_fp8(kMode) || ok) ok = mbar_wait(smem_u32(&sm->o_done), item_ctr & 1, abort_flag, p.err);
      if constexpr (is_fp8(kMode)) {  // the next piece starts at a shared barrier
        ok = !named_barrier_or(kDequantBarrier, 128 * kSoftmaxGroups, !ok);
        if (!ok) break;
      } else {
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
      }
      tc_fence_after();
      // (windowed: NaN sums, from a key that is not finite, stay NaN; they are no empty row)
      const bool has = kWindow ? !(lsum <= 0.f || bsum <= 0.f) : lsum > 0.f && bsum > 0.f;
      const bool final_out = pc.whole();
      float inv_l = has ? 1.f / bsum : 0.f;
      const float lse_v = has ? (m_use + __log2f(lsum)) * 0.69314718055994531f : NEG_INF;
      // attention sink: applied here to a final row, by the combine to a split row
      const int row0 = hb * kRowsPerCta + R * g;        // first query row of this warpgroup
      const int head0 = kWindow ? row0 % p.h : row0;    // and its head
      const int n_rows = kWindow ? pc.rows() : p.h;
      if (p.attn_sink && final_out && row0 + row < n_rows)
        inv_l *= attn_sink_factor(lse_v, p.attn_sink[head0 + row]);
      if (lane < R) bc_a[lane] = inv_l;
      __syncwarp();
      const volatile float* il = bc_a;  // 1 / sum of row i, read per store (broadcast)
      const int64_t ws_row0 = pc.split_row() * (kWindow ? p.n_hblk * kRowsPerCta : p.h) + row0;
      const int b = q / p.s_q, j = q % p.s_q + (kWindow ? row0 / p.h : 0);
      // h is a multiple of 16, so a warpgroup's 16 rows are all heads or all padding
      if (row0 < n_rows) {
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
          float o[R];  // O^T rows d of block m, columns = this warpgroup's 16 query rows
          tmem_ld16(t_o + 64 * m, o);
          tmem_wait_ld();
          const int d = 128 * m + 32 * wq + lane;
          // a row without keys (il = 0) is written as exact zeros: its O may
          // hold products of zero weights with rows nobody named
          if (final_out) {
            __nv_bfloat16* dst = p.out + (static_cast<int64_t>(q) * p.h + row0) * kDv + d;
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const float f = il[i];
              dst[i * kDv] = __float2bfloat16_rn(f != 0.f ? o[i] * f : 0.f);
            }
          } else {
            float* dst = p.ws_o + ws_row0 * kDv + d;
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const float f = il[i];
              dst[i * kDv] = f != 0.f ? o[i] * f : 0.f;
            }
          }
        }
      }
      if (wq == 0 && lane < R && row0 + lane < n_rows) {
        if (final_out)
          p.lse[(static_cast<int64_t>(b) * p.h + head0 + lane) * p.s_q + j] = lse_v;
        else
          p.ws_lse[ws_row0 + lane] = lse_v;
      }
      ++item_ctr;
    }
  }

  // ---- teardown
  if constexpr (kWindow) {  // a wait has failed: roles that left their loops
    if (__any_sync(0xffffffffu, *abort_flag != 0u) && (warp < kProducerWarp || lane == 0)) walk_list_out(p);
  }
  tc_fence_before();
  __syncthreads();
  // (after an abort: what this CTA left in flight, then what the peer did)
  if (*abort_flag) settle_after_abort();
  if (share) {
    cluster_sync();  // no peer still writes into this CTA's smem
    if (*abort_flag) settle_after_abort();
  }
  if (!kWindow) pdl_launch_dependents();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace mla
