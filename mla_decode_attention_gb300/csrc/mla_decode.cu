// Host entry points of the split-KV decode: argument checks, the launch of the
// split kernel and the PDL launch of the combine.
#include "mla_decode.h"
#include "mla_internal.h"
#include "mla_launch.cuh"

using namespace mla;

extern "C" int mla_decode_splitkv(const void* q, const void* kv_cache, int kv_format,
                                  int64_t num_pages, const int32_t* block_table,
                                  int64_t block_table_stride, const int32_t* cache_seqlens,
                                  int batch, int s_q, int h_q, float softmax_scale, int causal,
                                  const void* metadata, int num_sm_parts, void* workspace,
                                  void* out, float* lse, uint32_t* err, cudaStream_t stream) {
  int rc = check_common(batch, s_q, h_q, num_sm_parts);
  if (rc != MLA_OK) return rc;
  if (!q || !kv_cache || !block_table || !cache_seqlens || !metadata || !workspace || !out || !lse)
    return MLA_ERR_NULL;
  if (kv_format != MLA_KV_BF16 && kv_format != MLA_KV_FP8_656 && kv_format != MLA_KV_FP8_528)
    return MLA_ERR_UNSUPPORTED;
  if (num_pages <= 0 || num_pages > (int64_t{1} << 25) || block_table_stride <= 0)
    return MLA_ERR_SHAPE;
  if (!(softmax_scale > 0.f) || !(softmax_scale < 1e30f)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(metadata) || !aligned16(workspace) ||
      !aligned16(out))
    return MLA_ERR_ALIGN;

  const int n_seq = batch * s_q;
  const int n_hblk = head_blocks(h_q);
  const int rows = h_q < kRowsPerCta ? h_q : kRowsPerCta;
  // the V4.1 cache holds 512-wide keys (values are the whole key), others 576
  const int d_qk = kv_format == MLA_KV_FP8_528 ? kV41HeadDim : kDqk;

  SplitParams prm = {};
  prm.meta = static_cast<const int32_t*>(metadata);
  prm.block_table = block_table;
  prm.bt_stride = block_table_stride;
  prm.bt_width = block_table_stride;
  prm.num_pages = num_pages;
  prm.cache_seqlens = cache_seqlens;
  prm.causal = causal ? 1 : 0;
  prm.batch = batch;
  prm.topk = 0;
  prm.kv_rows = static_cast<const __nv_bfloat16*>(kv_cache);
  prm.kv_fp8 = static_cast<const uint8_t*>(kv_cache);
  prm.q = static_cast<const __nv_bfloat16*>(q);
  const int64_t ws_rows = workspace_rows(batch, s_q, num_sm_parts) * h_q;
  prm.ws_o = static_cast<float*>(workspace);
  prm.ws_lse = prm.ws_o + ws_rows * kDv;
  prm.ws_ctrl = workspace_ctrl(workspace, ws_rows);
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.lse = lse;
  prm.err = err;
  prm.h = h_q;
  prm.d_qk = d_qk;
  prm.s_q = s_q;
  prm.num_parts = num_sm_parts;
  prm.n_hblk = n_hblk;
  prm.rows = rows;
  prm.scale_log2 = softmax_scale * 1.4426950408889634f;
  CacheMaps maps;
  rc = make_cache_maps(&maps, prm, kv_cache, kv_format, h_q == pair::kRows);
  if (rc != MLA_OK) return rc;
  if (kv_format == MLA_KV_FP8_528)
    return launch_split<KvMode::kPagedFp8V41>(maps.q, maps.kv, prm, stream, &maps.codes, &maps.scales);
  if (kv_format == MLA_KV_FP8_656)
    return launch_split<KvMode::kPagedFp8>(maps.q, maps.kv, prm, stream, &maps.codes, &maps.scales);
  // 128 query rows: the two-SM kernel (scores and softmax on one SM, P.V on the other)
  if (h_q == pair::kRows) return launch_pair<false>(maps.kv, maps.quad4, maps.quad3, prm, stream);
  return launch_split<KvMode::kPagedBf16>(maps.q, maps.kv, prm, stream);
}

extern "C" int mla_decode(const void* q, const void* kv_cache, int kv_format, int64_t num_pages,
                          const int32_t* block_table, int64_t block_table_stride,
                          const int32_t* cache_seqlens, int batch, int s_q, int h_q,
                          float softmax_scale, int causal, const void* metadata, int num_sm_parts,
                          void* workspace, void* out, float* lse, uint32_t* err,
                          cudaStream_t stream) {
  const int rc = mla_decode_splitkv(q, kv_cache, kv_format, num_pages, block_table,
                                    block_table_stride, cache_seqlens, batch, s_q, h_q,
                                    softmax_scale, causal, metadata, num_sm_parts, workspace, out,
                                    lse, err, stream);
  if (rc != MLA_OK) return rc;
  return launch_combine(metadata, batch, s_q, h_q, num_sm_parts, workspace, nullptr, out, lse, stream,
                        true);
}

extern "C" int mla_sparse_decode_splitkv(const void* q, const void* kv, int64_t s_kv,
                                         const int32_t* indices, int topk, int batch, int s_q,
                                         int h_q, float softmax_scale, const float* attn_sink,
                                         const void* metadata, int num_sm_parts, void* workspace, void* out,
                                         float* lse, uint32_t* err, cudaStream_t stream) {
  int rc = check_common(batch, s_q, h_q, num_sm_parts);
  if (rc != MLA_OK) return rc;
  if (!q || !kv || !indices || !metadata || !workspace || !out || !lse) return MLA_ERR_NULL;
  if (topk <= 0 || s_kv <= 0 || s_kv > (int64_t{1} << 31) - 1) return MLA_ERR_SHAPE;
  if (!(softmax_scale > 0.f) || !(softmax_scale < 1e30f)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(kv) || !aligned16(metadata) || !aligned16(workspace) ||
      !aligned16(out))
    return MLA_ERR_ALIGN;

  const int n_seq = batch * s_q;
  const int rows = h_q < kRowsPerCta ? h_q : kRowsPerCta;
  CUtensorMap tm_q, tm_kv;
  if (!make_rows_map(&tm_q, q, static_cast<uint64_t>(n_seq) * h_q, kDqk * 2, rows))
    return record_error("cuTensorMapEncodeTiled failed for q", MLA_ERR_CUDA);
  // one-row boxes: each tile::gather4 fetches four arbitrary pool rows
  if (!make_rows_map(&tm_kv, kv, static_cast<uint64_t>(s_kv), kDqk * 2, 1))
    return record_error("cuTensorMapEncodeTiled failed for kv", MLA_ERR_CUDA);

  SplitParams prm = {};
  prm.meta = static_cast<const int32_t*>(metadata);
  prm.batch = batch;
  prm.causal = 0;
  prm.indices = indices;
  prm.attn_sink = attn_sink;
  prm.topk = topk;
  prm.s_kv = s_kv;
  prm.kv_rows = static_cast<const __nv_bfloat16*>(kv);
  prm.q = static_cast<const __nv_bfloat16*>(q);
  const int64_t ws_rows = workspace_rows(batch, s_q, num_sm_parts) * h_q;
  prm.ws_o = static_cast<float*>(workspace);
  prm.ws_lse = prm.ws_o + ws_rows * kDv;
  prm.ws_ctrl = workspace_ctrl(workspace, ws_rows);
  prm.out = static_cast<__nv_bfloat16*>(out);
  prm.lse = lse;
  prm.err = err;
  prm.h = h_q;
  prm.d_qk = kDqk;
  prm.s_q = s_q;
  prm.num_parts = num_sm_parts;
  prm.n_hblk = head_blocks(h_q);
  prm.rows = rows;
  prm.scale_log2 = softmax_scale * 1.4426950408889634f;
  // 128 query rows: the two-SM kernel with gathered keys
  return h_q == pair::kRows ? launch_pair<true>(tm_kv, tm_kv, tm_kv, prm, stream)
                            : launch_split<KvMode::kSparseBf16>(tm_q, tm_kv, prm, stream);
}

extern "C" int mla_sparse_decode(const void* q, const void* kv, int64_t s_kv,
                                 const int32_t* indices, int topk, int batch, int s_q, int h_q,
                                 float softmax_scale, const float* attn_sink, const void* metadata,
                                 int num_sm_parts, void* workspace, void* out, float* lse,
                                 uint32_t* err, cudaStream_t stream) {
  const int rc = mla_sparse_decode_splitkv(q, kv, s_kv, indices, topk, batch, s_q, h_q,
                                           softmax_scale, attn_sink, metadata, num_sm_parts,
                                           workspace, out, lse, err, stream);
  if (rc != MLA_OK) return rc;
  return launch_combine(metadata, batch, s_q, h_q, num_sm_parts, workspace, attn_sink, out, lse, stream,
                        true);
}

// DSA sparse prefill through the sparse decode path, each query token a
// request of one token (q [s_q, h_q, 576] is [s_q, 1, h_q, 576], indices
// [s_q, 1, topk] is [s_q, 1, topk], out [s_q, h_q, 512] is [s_q, 1, h_q, 512],
// lse [s_q, h_q] is [s_q, h_q, 1]).
extern "C" int mla_sparse_prefill(const void* q, const void* kv, int64_t s_kv, const int32_t* indices,
                                  int topk, int s_q, int h_q, float softmax_scale, const float* attn_sink,
                                  const void* metadata, int num_sm_parts, void* workspace, void* out,
                                  float* lse, uint32_t* err, cudaStream_t stream) {
  return mla_sparse_decode(q, kv, s_kv, indices, topk, s_q, 1, h_q, softmax_scale, attn_sink, metadata,
                           num_sm_parts, workspace, out, lse, err, stream);
}
