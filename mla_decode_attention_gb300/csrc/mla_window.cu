// Host entry points of the windowed decode (mla_window.cuh): argument checks,
// how the work is laid out and cut, launches; and the merge of cut items.
#include "mla_decode.h"
#include "mla_internal.h"
#include "mla_launch.cuh"
#include "mla_window.cuh"

namespace mla {

namespace {

// Merge of the items that were cut, per query row
//   lse = ln sum_i e^lse_i,   out = sum_i e^(lse_i - lse) o_i,
// over the item's pieces (those that hold no tile were not written and are left
// out).  A cut item belongs to the part with its first tile, which ends inside
// it, so a part has at most one.  All there is to it is the latency of reads from
// L2, so the blocks are one wave, what does not hang on the lengths is worked out
// before the attention kernel ends, a warp reads kMergeBatch pieces of a row at
// once, and rows of many pieces are shared by two to eight warps.  (us a call; the
// same without a merge; with as many blocks as rows ask for, a warp or a whole
// block a row: 3 requests of 128 heads over 8192 keys of the 528-byte cache 34 /
// 29 / 41, 48 of 64 heads over 1000 of the 656-byte cache 36 / 31 / 40, 10 of 128
// heads over 2000 28 / 24 / 31, two tokens of 128 requests over 4096 280 / 265 /
// 286.  Three pieces at once: 29 instead of 28 at 10 requests; four waves: 33.)
constexpr int kMergeWarps = 8;
constexpr int kMergeThreads = 32 * kMergeWarps;
constexpr int kMergeBatch = 2;
constexpr int kMergeBlocksPerSm = 2;

// Parts that may own a cut item: part k * step for k below the count.
struct MergeOwners {
  int count, step;
};
MergeOwners merge_owners(const WindowPlan& w) {
  // every item cut into the same pieces, a part each: its first one
  if (w.lanes == 1 && w.fixed == 0 && w.tiles % w.per == 0) return {w.items, static_cast<int>(w.tiles / w.per)};
  return {w.parts, 1};
}

// kShare: warps per row.
template <int kShare>
__global__ void __launch_bounds__(kMergeThreads, kMergeBlocksPerSm)
    window_merge_kernel(const __grid_constant__ SplitParams p, int block_rows, int owner_step) {
  constexpr int kBlockRows = kMergeWarps / kShare;
  __shared__ float4 s_acc[kShare > 1 ? kMergeWarps : 1][kDv / 4];
  __shared__ float s_mx[kMergeWarps], s_sum[kMergeWarps];
  const WindowPlan& w = p.plan;
  const int part = blockIdx.x * owner_step, line = part % w.lanes, pl = part / w.lanes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp % kShare;
  const int64_t m = floordiv((pl + 1) * w.per - 1, w.tiles + w.fixed);
  const int64_t item = line + w.lanes * m;
  const int pieces = static_cast<int>(window_last_part(w, m) - pl) + 1;
  const bool owner = item < w.items && window_first_part(w, m) == pl && pieces > 1;
  const int b = static_cast<int>(item) / w.chunks, j0 = (static_cast<int>(item) - b * w.chunks) * w.group;
  const int rows = min(w.group, p.s_q - j0) * p.h;
  const int first = window_row(w, m, pl, line);  // block of the first piece; the others begin their parts
  // Waited for whether or not there is anything to merge: a grid whose blocks all
  // had nothing to do would otherwise be over before the attention kernel is, and
  // let the kernel after it start.  That one may begin now and waits for this
  // grid (1.5 to 3 us a call between back-to-back calls).
  pdl_wait_primary();
  pdl_launch_dependents();
  if (!owner) return;
  const int tiles = window_span(window_ends(p.cache_seqlens, p.new_lens, p.s_q, b, j0, w.group), p.window, p.sinks).tiles;
  if (tiles == 0) return;  // the walking part writes its rows
  // this warp's pieces are share, share + kShare, ...; the block of the
  // workspace that holds the i-th of them, -1 where it has no tile
  const int mine = (pieces - share + kShare - 1) / kShare;
  auto block_of = [&](int i) {
    if (i >= mine) return -1;
    const int at = share + i * kShare;
    if (tiles != w.tiles) {
      const WindowPiece piece = window_piece(w, m, pl + at, tiles);
      if (piece.t0 >= piece.t1) return -1;
    }
    return at == 0 ? first : 2 * ((pl + at) * w.lanes + line);
  };
  int block = block_of(lane);
  for (int r0 = blockIdx.y * kBlockRows; r0 < rows; r0 += gridDim.y * kBlockRows) {
    const int r = r0 + warp / kShare;
    const bool in = r < rows;
    // lane l has columns 4 l .. 4 l + 3 of each 128
    float mx = -INFINITY, sum = 0.f;
    float4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < mine; i0 += 32) {
      if (mine > 32) block = block_of(i0 + lane);
      const float l = in && block >= 0 ? p.ws_lse[static_cast<int64_t>(block) * block_rows + r] : -INFINITY;
      const int n = min(mine - i0, 32);
      float4 v[kMergeBatch][4];
      auto load = [&](int i) {
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
          const int at = __shfl_sync(0xffffffffu, block, (i + k) & 31);
          const bool real = in && i + k < n && at >= 0;
          const float4* src = reinterpret_cast<const float4*>(p.ws_o + (static_cast<int64_t>(at) * block_rows + r) * kDv) + lane;
#pragma unroll
          for (int c = 0; c < 4; ++c) v[k][c] = real ? src[32 * c] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      };
      load(0);
      const float mx_new = fmaxf(mx, warp_max_f32(l));
      const float ref = mx_new == -INFINITY ? 0.f : mx_new;
      const float keep = i0 == 0 ? 0.f : __expf(mx - ref);  // what was summed before, at the new reference
      mx = mx_new;
      const float e = __expf(l - ref);  // 0 for a piece that is left out
      float part_sum = e;
#pragma unroll
      for (int sh = 16; sh > 0; sh >>= 1) part_sum += __shfl_xor_sync(0xffffffffu, part_sum, sh);
      sum = sum * keep + part_sum;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[c].x *= keep; acc[c].y *= keep; acc[c].z *= keep; acc[c].w *= keep;
      }
      for (int i = 0; i < n; i += kMergeBatch) {
        if (i > 0) load(i);
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
          const float f = i + k < n ? __shfl_sync(0xffffffffu, e, (i + k) & 31) : 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            acc[c].x += f * v[k][c].x; acc[c].y += f * v[k][c].y; acc[c].z += f * v[k][c].z; acc[c].w += f * v[k][c].w;
          }
        }
      }
    }
    if constexpr (kShare > 1) {  // the row's warps' sums, at the row's reference
      if (lane == 0) s_mx[warp] = mx;
      __syncthreads();
      const int w0 = warp - share;
      float top = s_mx[w0];
#pragma unroll
      for (int i = 1; i < kShare; ++i) top = fmaxf(top, s_mx[w0 + i]);
      const float f = mx == -INFINITY ? 0.f : __expf(mx - top);
      if (lane == 0) s_sum[warp] = sum * f;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        s_acc[warp][lane + 32 * c] = make_float4(acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f);
      __syncthreads();
      mx = top;
      sum = s_sum[w0];
#pragma unroll
      for (int i = 1; i < kShare; ++i) sum += s_sum[w0 + i];
    }
    const bool none = sum <= 0.f;  // (a NaN sum, from a key that is not finite, stays NaN)
    const float lse = none ? -INFINITY : mx + __logf(sum);
    float inv = none ? 0.f : 1.f / sum;
    const int j = j0 + r / p.h, head = r % p.h;
    if (p.attn_sink && in) inv *= attn_sink_factor(lse, p.attn_sink[head]);
    const int64_t tok = static_cast<int64_t>(b) * p.s_q + j;
    uint2* dst = reinterpret_cast<uint2*>(p.out + (tok * p.h + head) * kDv);
    if constexpr (kShare > 1) {
      for (int c = 32 * share + lane; c < kDv / 4 && in; c += 32 * kShare) {
        float4 v = s_acc[warp - share][c];
#pragma unroll
        for (int i = 1; i < kShare; ++i) {
          const float4 x = s_acc[warp - share + i][c];
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
        }
        dst[c] = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
      }
      __syncthreads();  // the next row's sums
    } else if (in) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        dst[lane + 32 * c] = make_uint2(pack_bf16x2(acc[c].x * inv, acc[c].y * inv), pack_bf16x2(acc[c].z * inv, acc[c].w * inv));
    }
    if (in && share == 0 && lane == 0) p.lse[(static_cast<int64_t>(b) * p.h + head) * p.s_q + j] = lse;
  }
}

int check_window(int batch, int s_q, int h_q, int window, int sinks, int num_sm_parts) {
  if (batch <= 0 || s_q <= 0 || static_cast<int64_t>(batch) * s_q > (1 << 24)) return MLA_ERR_SHAPE;
  if (!heads_supported(h_q) || window <= 0 || sinks < 0 || num_sm_parts <= 0 || num_sm_parts > (1 << 20))
    return MLA_ERR_SHAPE;
  return MLA_OK;
}

// Which kernel a call runs on, and its plan.  The two-SM kernel takes 128 query
// rows and the bf16 cache; the one-SM kernel 64 rows (two CTAs for 128 heads)
// and every cache.  Fewer heads than rows: tokens of a request fill the block.
// A bf16 call goes to the two-SM kernel when a block of it gets more rows than
// a block of the other would hold.
struct WindowCall {
  bool pair;
  int block_rows;  // query rows of a block = rows of a workspace block
  WindowPlan plan;
};
// Fixed cost of a piece, and cost of a merge to the call, in tiles, from sweeps of
// both (us, cut by this rule / never cut):
//   two-SM kernel   128 requests x 2 tokens x 128 heads over 4096   280 / 295
//                   85 requests of 128 heads over 8192  267 / 298;  160 x 128 over 8192  465 / 534
//                   10 x 128 over 2000  28 / 43
//   one-SM kernel   200 requests of 64 heads over 4096  226 / 307;  160 x 64 over 2000
//                   104 / 164;  656-byte cache, 100 x 128 over 2000  168 / 226
// and where a merge at 4 tiles would have cut and lost: 90 requests of 128 heads
// over 1000 keys 60 cut, 54 whole.
constexpr int kPairFixed = 5, kPairMerge = 6, kOneFixed = 2, kOneMerge = 1;

WindowCall window_call(int batch, int s_q, int h_q, int window, int sinks, int num_sm_parts, bool bf16, bool ragged) {
  WindowCall c;
  const int sms = num_sm_parts * head_blocks(h_q);  // SMs that the parts stand for
  const int most = pair::kRows / h_q;
  const int fill = (s_q < most ? s_q : most) * h_q;
  c.pair = bf16 && fill > kRowsPerCta;
  c.block_rows = c.pair || h_q > kRowsPerCta ? pair::kRows : kRowsPerCta;
  const int tokens = c.block_rows / h_q;
  const int parts = c.pair ? (sms > 1 ? sms / 2 : 1) : num_sm_parts;
  c.plan = window_plan(batch, s_q, s_q < tokens ? s_q : tokens, window, sinks, parts, ragged,
                       c.pair ? kPairFixed : kOneFixed, c.pair ? kPairMerge : kOneMerge);
  return c;
}

// Two blocks of partial rows per part, as many rows whichever kernel runs.
size_t window_bytes(const WindowCall& c) {
  return c.plan.whole ? 0 : static_cast<size_t>(2) * c.plan.parts * c.block_rows * (kDv + 1) * sizeof(float);
}

}  // namespace

}  // namespace mla

using namespace mla;

extern "C" int mla_window_workspace_size(int batch, int s_q, int h_q, int window, int sinks, int num_sm_parts,
                                         size_t* bytes) {
  if (!bytes) return MLA_ERR_NULL;
  const int rc = check_window(batch, s_q, h_q, window, sinks, num_sm_parts);
  if (rc != MLA_OK) return rc;
  // the call may be with either kind of cache, with or without new_lens
  size_t most = 0;
  for (int bf16 = 0; bf16 < 2; ++bf16) {
    const size_t n = window_bytes(window_call(batch, s_q, h_q, window, sinks, num_sm_parts, bf16 != 0, false));
    most = n > most ? n : most;
  }
  *bytes = most;
  return MLA_OK;
}

extern "C" int mla_window_decode(const void* q, const void* kv_cache, int kv_format, int64_t num_pages,
                                 const int32_t* block_table, int64_t block_table_stride, int64_t max_pages,
                                 const int32_t* cache_seqlens, const int32_t* new_lens, int batch, int s_q, int h_q,
                                 int window, int sinks, float softmax_scale, const float* attn_sink, int num_sm_parts,
                                 void* workspace, size_t workspace_bytes, void* out, float* lse, uint32_t* err,
                                 cudaStream_t stream) {
  int rc = check_window(batch, s_q, h_q, window, sinks, num_sm_parts);
  if (rc != MLA_OK) return rc;
  if (!q || !kv_cache || !block_table || !cache_seqlens || !out || !lse) return MLA_ERR_NULL;
  if (kv_format != MLA_KV_BF16 && kv_format != MLA_KV_FP8_656 && kv_format != MLA_KV_FP8_528)
    return MLA_ERR_UNSUPPORTED;
  if (num_pages <= 0 || num_pages > (int64_t{1} << 25) || max_pages <= 0 ||
      (batch > 1 && block_table_stride < max_pages))
    return MLA_ERR_SHAPE;
  if (!(softmax_scale > 0.f) || !(softmax_scale < 1e30f)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(workspace) || !aligned16(out)) return MLA_ERR_ALIGN;

  const WindowCall call = window_call(batch, s_q, h_q, window, sinks, num_sm_parts, kv_format == MLA_KV_BF16,
                                      new_lens != nullptr);
  const size_t need = window_bytes(call);
  if (need > 0 && !workspace) return MLA_ERR_NULL;
  if (need > workspace_bytes) return record_error("mla_window_decode: the workspace is too small", MLA_ERR_SHAPE);
  SplitParams prm = {};
  prm.block_table = block_table;
  prm.bt_stride = block_table_stride;
  prm.bt_width = max_pages;
  prm.num_pages = num_pages;
  prm.cache_seqlens = cache_seqlens;
  prm.new_lens = new_lens;
  prm.window = window;
  prm.sinks = sinks;
  prm.plan = call.plan;
  prm.batch = batch;
  prm.attn_sink = attn_sink;
  prm.kv_rows = static_cast<const __nv_bfloat16*>(kv_cache);
  prm.kv_fp8 = static_cast<const uint8_t*>(kv_cache);
  prm.q = static_cast<const __nv_bfloat16*>(q);
  prm.ws_o = static_cast<float*>(workspace);
  if (need > 0) prm.ws_lse = prm.ws_o + static_cast<int64_t>(2) * call.plan.parts * call.block_rows * kDv;
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.lse = lse;
  prm.err = err;
  prm.h = h_q;
  prm.d_qk = kv_format == MLA_KV_FP8_528 ? kV41HeadDim : kDqk;
  prm.s_q = s_q;
  prm.num_parts = call.plan.parts;
  prm.n_hblk = head_blocks(h_q);
  prm.rows = h_q > kRowsPerCta ? kRowsPerCta : (call.pair ? kRowsPerCta : call.plan.group * h_q);
  prm.scale_log2 = softmax_scale * 1.4426950408889634f;

  CacheMaps maps;
  rc = make_cache_maps(&maps, prm, kv_cache, kv_format, call.pair);
  if (rc != MLA_OK) return rc;
  if (kv_format == MLA_KV_FP8_528)
    rc = launch_split<KvMode::kPagedFp8V41, true>(maps.q, maps.kv, prm, stream, &maps.codes, &maps.scales);
  else if (kv_format == MLA_KV_FP8_656)
    rc = launch_split<KvMode::kPagedFp8, true>(maps.q, maps.kv, prm, stream, &maps.codes, &maps.scales);
  else if (call.pair)
    rc = launch_pair<false, true>(maps.kv, maps.quad4, maps.quad3, prm, stream);
  else
    rc = launch_split<KvMode::kPagedBf16, true>(maps.q, maps.kv, prm, stream);
  if (rc != MLA_OK || call.plan.whole) return rc;

  cudaLaunchConfig_t cfg = {};
  const MergeOwners owners = merge_owners(call.plan);
  const int64_t pieces = owners.step > 1 ? owners.step : (call.plan.tiles + call.plan.per - 1) / call.plan.per + 1;
  const int rows = call.plan.group * h_q;
  const int64_t blocks = static_cast<int64_t>(kMergeBlocksPerSm) * num_sm_parts * head_blocks(h_q);  // one wave
  // as many warps a row as one batch of pieces each takes, while there are any
  int share = 1;
  while (share < kMergeWarps && share * kMergeBatch < pieces &&
         2 * share * static_cast<int64_t>(rows) * owners.count <= blocks * kMergeWarps)
    share *= 2;
  const int64_t lines = (static_cast<int64_t>(rows) * share + kMergeWarps - 1) / kMergeWarps;
  const int64_t fit = blocks / owners.count;
  cfg.gridDim = dim3(owners.count, static_cast<unsigned>(lines < fit ? lines : (fit > 1 ? fit : 1)), 1);
  cfg.blockDim = dim3(kMergeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* kernel = share == 1   ? window_merge_kernel<1>
                 : share == 2 ? window_merge_kernel<2>
                 : share == 4 ? window_merge_kernel<4>
                              : window_merge_kernel<8>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm, call.block_rows, owners.step);
  return e == cudaSuccess ? MLA_OK : record_cuda_error("window merge kernel launch", e);
}
