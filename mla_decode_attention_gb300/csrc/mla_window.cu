// Host entry points of the windowed decode (mla_window.cuh): argument checks,
// the number of pieces a token's tiles are cut into, launches.
#include "mla_decode.h"
#include "mla_internal.h"
#include "mla_launch.cuh"
#include "mla_window.cuh"

namespace mla {

namespace {

// Pieces per token.  Every token has at most `tiles` tiles; a piece costs its
// tiles plus kFixedCost (query load, epilogue), and cutting costs the fp32
// partial rows and the combine besides, about kSplitCost tiles.  With few
// tokens the parts would otherwise idle.
constexpr int kSplitCost = 2;
int window_splits(int64_t n_seq, int tiles, int parts) {
  int best = 1;
  int64_t best_cost = 0;
  for (int n = 1; n <= tiles && n <= 2 * parts; ++n) {
    const int64_t rounds = (n_seq * n + parts - 1) / parts;
    const int64_t cost = rounds * ((tiles + n - 1) / n + kFixedCost) + (n > 1 ? kSplitCost : 0);
    if (n == 1 || cost < best_cost) {
      best = n;
      best_cost = cost;
    }
    if (n_seq * n >= 2 * static_cast<int64_t>(parts)) break;  // every part has work: more pieces only cost
  }
  return best;
}

int check_window(int batch, int s_q, int h_q, int window, int sinks, int num_sm_parts) {
  if (batch <= 0 || s_q <= 0 || static_cast<int64_t>(batch) * s_q > (1 << 24)) return MLA_ERR_SHAPE;
  if (!heads_supported(h_q) || window <= 0 || sinks < 0 || num_sm_parts <= 0) return MLA_ERR_SHAPE;
  return MLA_OK;
}

}  // namespace

}  // namespace mla

using namespace mla;

extern "C" int mla_window_workspace_size(int batch, int s_q, int h_q, int window, int sinks, int num_sm_parts,
                                         size_t* bytes) {
  if (!bytes) return MLA_ERR_NULL;
  const int rc = check_window(batch, s_q, h_q, window, sinks, num_sm_parts);
  if (rc != MLA_OK) return rc;
  const int64_t n_seq = static_cast<int64_t>(batch) * s_q;
  const int n_split = window_splits(n_seq, window_max_tiles(window, sinks), num_sm_parts);
  *bytes = n_split == 1 ? 0 : static_cast<size_t>(n_seq) * n_split * h_q * (kDv + 1) * sizeof(float);
  return MLA_OK;
}

extern "C" int mla_window_decode(const void* q, const void* kv_cache, int kv_format, int64_t num_pages,
                                 const int32_t* block_table, int64_t block_table_stride, int64_t max_pages,
                                 const int32_t* cache_seqlens, const int32_t* new_lens, int batch, int s_q, int h_q,
                                 int window, int sinks, float softmax_scale, const float* attn_sink, int num_sm_parts,
                                 void* workspace, void* out, float* lse, uint32_t* err, cudaStream_t stream) {
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

  const int n_seq = batch * s_q;
  const int n_split = window_splits(n_seq, window_max_tiles(window, sinks), num_sm_parts);
  if (n_split > 1 && !workspace) return MLA_ERR_NULL;
  SplitParams prm = {};
  prm.block_table = block_table;
  prm.bt_stride = block_table_stride;
  prm.bt_width = max_pages;
  prm.num_pages = num_pages;
  prm.cache_seqlens = cache_seqlens;
  prm.new_lens = new_lens;
  prm.window = window;
  prm.sinks = sinks;
  prm.n_split = n_split;
  prm.batch = batch;
  prm.attn_sink = attn_sink;
  prm.kv_rows = static_cast<const __nv_bfloat16*>(kv_cache);
  prm.kv_fp8 = static_cast<const uint8_t*>(kv_cache);
  prm.q = static_cast<const __nv_bfloat16*>(q);
  prm.ws_o = static_cast<float*>(workspace);
  prm.ws_lse = prm.ws_o + static_cast<int64_t>(n_seq) * n_split * h_q * kDv;
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.lse = lse;
  prm.err = err;
  prm.h = h_q;
  prm.d_qk = kv_format == MLA_KV_FP8_528 ? kV41HeadDim : kDqk;
  prm.s_q = s_q;
  prm.num_parts = num_sm_parts;
  prm.n_hblk = head_blocks(h_q);
  prm.rows = h_q < kRowsPerCta ? h_q : kRowsPerCta;
  prm.scale_log2 = softmax_scale * 1.4426950408889634f;

  CacheMaps maps;
  rc = make_cache_maps(&maps, prm, kv_cache, kv_format);
  if (rc != MLA_OK) return rc;
  if (kv_format == MLA_KV_FP8_528)
    rc = launch_split<KvMode::kPagedFp8V41, true>(maps.q, maps.kv, prm, stream, &maps.codes, &maps.scales);
  else if (kv_format == MLA_KV_FP8_656)
    rc = launch_split<KvMode::kPagedFp8, true>(maps.q, maps.kv, prm, stream, &maps.codes, &maps.scales);
  else if (h_q == pair::kRows)
    rc = launch_pair<false, true>(maps.kv, maps.quad4, maps.quad3, prm, stream);
  else
    rc = launch_split<KvMode::kPagedBf16, true>(maps.q, maps.kv, prm, stream);
  if (rc != MLA_OK || n_split == 1) return rc;
  return launch_window_combine(cache_seqlens, new_lens, batch, s_q, h_q, window, sinks, n_split, workspace, attn_sink,
                               out, lse, stream);
}
