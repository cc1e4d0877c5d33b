// Entry points of the attention of packed sequences (mla_prefill.cuh).
#include <algorithm>

#include "mla_host.cuh"
#include "mla_merge.cuh"
#include "mla_prefill.cuh"

namespace mla {

namespace {

using prefill::kKeys;
using prefill::kNope;
using prefill::kRope;
using prefill::kRows;
using prefill::kValue;

// Pieces that each block of query rows' keys are cut into.  Known without the lengths, so that a
// workspace fits whatever they are, and of kLeastTiles key tiles at least on average.
//
// Several sequences differ in length.  Where their blocks are fewer than SMs: up to three pieces an SM, which go
// to whoever is free (3 sequences over 8000 to 16384 keys, 16 heads: 69 us with one an SM, 64
// so, 67 with four), or none: whole, the call takes as long as its longest block; cut, as its pieces on
// all SMs and a quarter of the longest at the end.  In key tiles, a piece costs 1.5 with few rows and 3.5 with all 256,
// a launch 4, the merge 2.  (us whole and in 2, 3, 4 pieces, causal: 2 of 2048 tokens, 8 heads, 41, 45, 47, 53; 2 of
// 1024, 16 heads, 24, 35, 40, 46; over 2048 keys 42, 50, 53, 58; 2 of 4096, 4 heads, 75, 58, 57, 63; 16 tokens over
// 1000 keys each, 4 heads, 16.8, 14.7, 17.6, 17.2; over 4000, 8 heads, 53, 57, 58, 58; 2 of 100 over 1500, 8 heads, 22,
// 17, 14, 13.)
//
// Otherwise what costs least by this count in key tiles: a piece costs its share of the keys and, cut, its
// query rows, its fp32 rows and their merge, 1.5 tiles with few rows and 5 with all 256; a merge's launch costs 2.  Pieces
// of one sequence end together, so they run in whole rounds; those of several fill
// the gaps but for half of a long one at the end.  (us for 1, 2, 3, 4, 6, 8 pieces, 40 heads of 1024 over 9024 keys: 260,
// 215, 197, 192, 197, 207; 200 heads of 100 over 12100: 287, 229, 220, 241, 236, 247; 128 heads of 512 over 16512:
// 535, 572, 563, 529, 537, 549; 20 heads of 2048 over themselves: 42, 51, 57, 64; 2 sequences of 300
// over 16300, 40 heads: 448, 305, 289, 275, 271, 275.)
//
// Pieces take a workspace: 516 bytes for each of their rows.  So they are made only where they save a thirtieth by
// this count (the saving of thousands of blocks is less than its error: 8192 tokens of 128 heads over 262144 keys, two
// sequences, two pieces for 0.5 % and 1.1 GB), and their rows are those of eight full blocks an SM at most, 160 MB on 152.
constexpr int kLeastTiles = 2, kMostSplits = 32;
constexpr int64_t kMostPartialRows = 8 * 2 * kRows;  // for each SM
constexpr double kWorth = 29. / 30.;
int splits_of(int64_t total_q, int64_t total_k, int batch, int h_q, int h_k, int num_sm_parts) {
  const int64_t per = 2 * (kRows / (h_q / h_k));
  const int64_t blocks = (total_q + batch * (per - 1)) / per * h_k;
  if (total_q == 0) return 1;
  const int64_t tiles = total_k / batch / kKeys, sms = std::min(num_sm_parts, 1 << 16);
  const int64_t most = std::clamp<int64_t>(sms * kMostPartialRows / (total_q * h_q), 1, kMostSplits);
  // (a causal call's mean; without a mask rows have up to twice as many)
  const double mean = static_cast<double>(std::max(total_k - total_q / 2, total_k / 2)) / batch / kKeys;
  const double full = static_cast<double>(total_q * h_q) / static_cast<double>(blocks * 2 * kRows);
  if (batch > 1 && blocks <= sms) {
    const int64_t up_to = std::max(std::min(sms / blocks, tiles / kLeastTiles), std::min(3 * sms / blocks, tiles / (2 * kLeastTiles)));
    const int s = static_cast<int>(std::clamp<int64_t>(up_to, 1, most));
    const double piece = 1.5 + 2. * full, length = static_cast<double>(total_k) / batch / kKeys, longest = length / s + piece;
    const double cut = 6. + std::max(longest, (mean / s + piece) * s * blocks / sms + 0.25 * longest);
    return cut < kWorth * (5. + length) ? s : 1;
  }
  const double piece = 1.5 + 3.5 * full;
  int best = 1;
  double least = 0.;
  for (int s = 1; s <= std::clamp<int64_t>(tiles / kLeastTiles, 1, most); ++s) {
    const double each = s == 1 ? mean + 1. : mean / s + piece, launch = s == 1 ? 0. : 2.;
    const int64_t rounds = (blocks * s + sms - 1) / sms;
    const double cost = launch + (batch == 1 ? rounds * each : each * s * blocks / sms + 0.75 * mean / s);
    if (s == 1 || cost < least) {
      least = s == 1 ? kWorth * cost : cost;
      best = s;
    }
  }
  return best;
}

int check_sizes(int64_t total_q, int64_t total_k, int batch, int h_q, int h_k, int num_sm_parts) {
  if (batch <= 0 || batch > kMaxSequences || total_q < 0 || total_q > kMaxPackedRows || total_k < 0 || total_k > kMaxPackedRows)
    return MLA_ERR_SHAPE;
  // (the kernel counts blocks of query rows in 32 bits)
  if (h_q <= 0 || h_k <= 0 || h_q % h_k != 0 || h_q / h_k > kRows || h_q > (1 << 16) || num_sm_parts <= 0) return MLA_ERR_SHAPE;
  const int64_t per = 2 * (kRows / (h_q / h_k));
  if (((total_q + batch * (per - 1)) / per * h_k) > (int64_t{1} << 26)) return MLA_ERR_SHAPE;
  return MLA_OK;
}

// A bf16 tensor of `n` dimensions with 64-column rows in the first, `strides` elements
// apart in the others; boxes of `box` rows with 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int n, const int64_t* dims, const int64_t* strides, const int* box) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[5] = {64u}, st[4];
  cuuint32_t b[5] = {64u};
  const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
  for (int i = 0; i < n; ++i) {
    d[i + 1] = static_cast<cuuint64_t>(dims[i]);
    st[i] = static_cast<cuuint64_t>(strides[i]) * 2u;
    b[i + 1] = static_cast<cuuint32_t>(box[i]);
  }
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(n + 1), const_cast<void*>(base), d, st, b, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows as [tokens][key heads][group][chunks][64]: boxes of a chunk of `box` tokens
// of a key head's group, which land token by token.
bool make_query_map(CUtensorMap* m, const void* base, int cols, int group, int h_k, int64_t tokens, int64_t head, int64_t token, int box_tokens) {
  const int64_t dims[4] = {group, tokens, cols / 64, h_k}, strides[4] = {head, token, 64, head * group};
  const int box[4] = {group, box_tokens, 1, 1};
  return make_map(m, base, 4, dims, strides, box);
}

// Keys or values as [heads][2 chunks][tokens][64]: boxes of `chunks` chunks of 128 tokens of a head.
bool make_key_map(CUtensorMap* m, const void* base, int heads, int64_t tokens, int64_t head, int64_t token, int chunks) {
  const int64_t dims[3] = {tokens, 2, heads}, strides[3] = {token, 64, head};
  const int box[3] = {kKeys, chunks, 1};
  return make_map(m, base, 3, dims, strides, box);
}

// Position columns as [heads][1 chunk][tokens][64].
bool make_rope_map(CUtensorMap* m, const void* base, int heads, int64_t tokens, int64_t head, int64_t token) {
  const int64_t dims[3] = {tokens, 1, heads}, strides[3] = {token, 64, head};
  const int box[3] = {kKeys, 1, 1};
  return make_map(m, base, 3, dims, strides, box);
}

template <bool kHasRope>
int launch_prefill(const prefill::Maps& maps, const prefill::Params& p, int64_t blocks, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};  // per instantiation
  const int rc = allow_shared_memory(prefill::mla_prefill_kernel<kHasRope>, prefill::kSmemBytes, &done,
                                     "cudaFuncSetAttribute(prefill kernel)");
  if (rc != MLA_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(prefill::kThreads, 1, 1);
  cfg.dynamicSmemBytes = prefill::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, prefill::mla_prefill_kernel<kHasRope>, maps, p);
  return e == cudaSuccess ? MLA_OK : record_cuda_error("prefill kernel launch", e);
}

// Strides that TMA takes: whole 16-byte units, rows that do not begin before the
// last has ended (a dimension of one has none).
bool stride_ok(int64_t stride, int64_t count, int64_t width) {
  return count <= 1 || (stride >= width && stride <= kMaxTokenStride);
}

}  // namespace

}  // namespace mla

using namespace mla;

extern "C" int mla_prefill_workspace_size(int64_t total_q, int64_t total_k, int batch, int h_q, int h_k, int num_sm_parts,
                                          size_t* bytes) {
  if (!bytes) return MLA_ERR_NULL;
  const int rc = check_sizes(total_q, total_k, batch, h_q, h_k, num_sm_parts);
  if (rc != MLA_OK) return rc;
  const int splits = splits_of(total_q, total_k, batch, h_q, h_k, num_sm_parts);
  *bytes = splits > 1 ? static_cast<size_t>(splits) * total_q * h_q * (kValue + 1) * sizeof(float) : 0;
  return MLA_OK;
}

extern "C" int mla_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k, int64_t k_token_stride,
                           int64_t k_head_stride, const void* k_rope, int64_t k_rope_token_stride, int64_t k_rope_head_stride,
                           const void* v, int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_k, int batch, int64_t total_q, int64_t total_k, int h_q, int h_k,
                           float softmax_scale, int causal, int num_sm_parts, void* workspace, size_t workspace_bytes, void* out,
                           int64_t out_token_stride, int64_t out_head_stride, float* lse, uint32_t* err, cudaStream_t stream) {
  const int rc = check_sizes(total_q, total_k, batch, h_q, h_k, num_sm_parts);
  if (rc != MLA_OK) return rc;
  if (!(softmax_scale > 0.f) || !(softmax_scale < 1e30f)) return MLA_ERR_SHAPE;
  if (total_q == 0) return MLA_OK;
  if (!q || !cu_seqlens_q || !cu_seqlens_k || !out || !lse || (total_k > 0 && (!k || !v))) return MLA_ERR_NULL;
  const int d_qk = k_rope ? kNope + kRope : kNope;
  if (!stride_ok(q_token_stride, total_q, d_qk) || !stride_ok(q_head_stride, h_q, d_qk) ||
      !stride_ok(k_token_stride, total_k, kNope) || !stride_ok(k_head_stride, h_k, kNope) ||
      !stride_ok(v_token_stride, total_k, kValue) || !stride_ok(v_head_stride, h_k, kValue) ||
      (k_rope && (!stride_ok(k_rope_token_stride, total_k, kRope) ||
                  (k_rope_head_stride != 0 && !stride_ok(k_rope_head_stride, h_k, kRope)))) ||
      out_token_stride > kMaxTokenStride || out_head_stride > kMaxTokenStride ||
      !rows_apart(total_q, h_q, out_token_stride, out_head_stride, kValue))
    return MLA_ERR_SHAPE;
  // a dimension of one has no stride of its own: any that TMA takes
  const auto st = [](int64_t stride, int64_t count, int64_t width) { return count > 1 ? stride : width; };
  const int64_t q_token = st(q_token_stride, total_q, 192), q_head = st(q_head_stride, h_q, 192);
  const int64_t k_token = st(k_token_stride, total_k, kNope), k_head = st(k_head_stride, h_k, kNope);
  const int64_t v_token = st(v_token_stride, total_k, kValue), v_head = st(v_head_stride, h_k, kValue);
  const bool rope_per_head = k_rope && k_rope_head_stride != 0 && h_k > 1;
  const int64_t rope_token = st(k_rope_token_stride, total_k, kRope), rope_head = rope_per_head ? k_rope_head_stride : kRope;
  const int64_t out_token = st(out_token_stride, total_q, kValue), out_head = st(out_head_stride, h_q, kValue);
  const int64_t strides = q_token | q_head | k_token | k_head | v_token | v_head | out_token | out_head | (k_rope ? rope_token | rope_head : 0);
  if (!aligned16(q) || !aligned16(k) || !aligned16(k_rope) || !aligned16(v) || !aligned16(out) || !aligned32(workspace) ||
      strides % 8 != 0)
    return MLA_ERR_ALIGN;
  const int splits = splits_of(total_q, total_k, batch, h_q, h_k, num_sm_parts);
  const int64_t ws_rows = static_cast<int64_t>(splits) * total_q * h_q;
  if (splits > 1) {
    if (!workspace) return MLA_ERR_NULL;
    if (workspace_bytes < static_cast<size_t>(ws_rows) * (kValue + 1) * sizeof(float)) return MLA_ERR_SHAPE;
  }

  const int group = h_q / h_k, tokens = kRows / group;
  prefill::Maps maps;
  bool ok = make_query_map(&maps.q, q, d_qk, group, h_k, total_q, q_head, q_token, tokens);
  maps.k = maps.v = maps.rope = maps.k1 = maps.v1 = maps.q;  // (without keys not read: no item has a key tile)
  if (total_k > 0) {
    ok = ok && make_key_map(&maps.k, k, h_k, total_k, k_head, k_token, 2) && make_key_map(&maps.v, v, h_k, total_k, v_head, v_token, 2);
    if (k_rope)
      ok = ok && make_rope_map(&maps.rope, k_rope, rope_per_head ? h_k : 1, total_k, rope_head, rope_token) &&
           make_key_map(&maps.k1, k, h_k, total_k, k_head, k_token, 1) && make_key_map(&maps.v1, v, h_k, total_k, v_head, v_token, 1);
  }
  if (!ok) return record_error("cuTensorMapEncodeTiled failed for q, k, k_rope or v", MLA_ERR_CUDA);

  prefill::Params p = {};
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.batch = batch;
  p.total_q = static_cast<int>(total_q);
  p.total_k = static_cast<int>(total_k);
  p.h_k = static_cast<uint32_t>(h_k);
  p.group = group;
  p.tokens = tokens;
  p.per_inverse = ((uint64_t{1} << 38) + 2 * tokens - 1) / (2 * tokens);
  p.causal = causal != 0;
  p.rope_per_head = rope_per_head;
  p.splits = splits;
  p.parts = static_cast<uint32_t>(num_sm_parts < (1 << 16) ? num_sm_parts : (1 << 16));
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_token = out_token;
  p.out_head = out_head;
  p.out_wide = reinterpret_cast<uintptr_t>(out) % 32 == 0 && (out_token | out_head) % 16 == 0;
  p.lse = lse;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = splits > 1 ? p.ws_o + ws_rows * kValue : nullptr;
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.v_token = v_token;
  p.v_head = v_head;
  p.err = err;
  // as many blocks as items at most, whatever the lengths (a block that runs takes on further items)
  const int64_t per = 2 * tokens, blocks = (total_q + batch * (per - 1)) / per * h_k * splits;
  const int status = k_rope ? launch_prefill<true>(maps, p, blocks, stream) : launch_prefill<false>(maps, p, blocks, stream);
  if (status != MLA_OK || splits == 1) return status;

  merge::Params g = {};
  g.parts = p.ws_o;
  g.part_stride = total_q * h_q * kValue;
  g.token_stride = static_cast<int64_t>(h_q) * kValue;
  g.head_stride = kValue;
  g.lses = p.ws_lse;
  g.lse_part = h_q * total_q;
  g.lse_head = total_q;
  g.lse_token = 1;
  g.n = splits;
  g.heads = h_q;
  g.d = kValue;
  g.tokens = static_cast<uint32_t>(total_q);
  g.rows_from = cu_seqlens_q;           // rows of no sequence stay as they were
  g.rows_to = cu_seqlens_q + batch;
  g.out = p.out;
  g.out_token = out_token;
  g.out_head = out_head;
  g.lse = lse;
  g.out_lse_head = total_q;
  g.out_lse_token = 1;
  return merge::launch_type<true>(g, stream);
}
