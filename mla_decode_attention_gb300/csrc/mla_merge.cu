// Entry point of the merge of attention states (mla_merge.cuh).
#include "mla_merge.cuh"

using namespace mla;

extern "C" int mla_merge_states(const void* parts, int parts_fp32, int64_t part_stride, int64_t token_stride,
                                int64_t head_stride, const float* lses, int64_t lse_part_stride, int64_t lse_head_stride,
                                int64_t lse_token_stride, int n, int64_t tokens, int h_q, int d, void* out,
                                int64_t out_token_stride, int64_t out_head_stride, float* lse, int64_t out_lse_head_stride,
                                int64_t out_lse_token_stride, cudaStream_t stream) {
  if (n <= 0 || h_q <= 0 || tokens < 0 || d < 8 || d > 512 || d % 8 != 0) return MLA_ERR_SHAPE;
  if (tokens > (int64_t{1} << 31) / h_q) return MLA_ERR_SHAPE;  // (rows are counted in 32 bits)
  if (tokens == 0) return MLA_OK;
  if (!parts || !lses || !out || !lse) return MLA_ERR_NULL;
  for (const int64_t s : {part_stride, token_stride, head_stride, lse_part_stride, lse_head_stride, lse_token_stride,
                          out_token_stride, out_head_stride, out_lse_head_stride, out_lse_token_stride})
    if (s < 0 || s > kMaxTokenStride) return MLA_ERR_SHAPE;
  // rows of the output lie apart: heads within a token, or tokens within a head
  if (!rows_apart(tokens, h_q, out_token_stride, out_head_stride, d) ||
      !rows_apart(tokens, h_q, out_lse_token_stride, out_lse_head_stride, 1))
    return MLA_ERR_SHAPE;
  // a dimension of one has no stride of its own
  if (n == 1) part_stride = 0;
  if (tokens == 1) token_stride = out_token_stride = 0;
  if (h_q == 1) head_stride = out_head_stride = 0;
  const int unit = parts_fp32 ? 4 : 8;
  if (!aligned16(parts) || !aligned16(out) || part_stride % unit != 0 || token_stride % unit != 0 || head_stride % unit != 0 ||
      out_token_stride % 8 != 0 || out_head_stride % 8 != 0)
    return MLA_ERR_ALIGN;
  merge::Params p = {};
  p.parts = parts;
  p.part_stride = part_stride;
  p.token_stride = token_stride;
  p.head_stride = head_stride;
  p.lses = lses;
  p.lse_part = lse_part_stride;
  p.lse_head = lse_head_stride;
  p.lse_token = lse_token_stride;
  p.n = n;
  p.heads = h_q;
  p.d = d;
  p.tokens = static_cast<uint32_t>(tokens);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_token = out_token_stride;
  p.out_head = out_head_stride;
  p.lse = lse;
  p.out_lse_head = out_lse_head_stride;
  p.out_lse_token = out_lse_token_stride;
  return parts_fp32 ? merge::launch_type<true>(p, stream) : merge::launch_type<false>(p, stream);
}
