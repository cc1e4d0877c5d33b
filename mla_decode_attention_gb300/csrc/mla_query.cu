// RMS norm of every query head and rotation of its last 64 columns, one pass:
//   y = x * w / sqrt(mean(x^2) + eps)   (when eps > 0; over the head's d columns)
//   y[d-64 .. d) turned by the token's angles, rounded once to bf16.
//
// Bound by memory: every head is read once and written once.  Eight lanes own
// a head and hold all of it in registers (d / 64 units of 16 bytes a lane), so
// the norm's sum is three shuffles and no column is read twice.  2048 tokens of
// 128 heads: 512 columns normed 83 us = 6.5 TB/s (95 % of the copy rate), 576
// columns rotated alone, out of place, 88 us = 6.9 TB/s.  A decode step of 64
// tokens of 128 x 576 takes 2.9 us, its bytes at the copy rate 2.8.
#include "mla_rope.cuh"

namespace mla {

namespace {

// Small blocks, so that one's loads overlap its neighbours' sums (3000 tokens of
// 64 x 512: 61.5 us; 65 with 256 threads, 79 with 512).
constexpr int kQueryThreads = 128;

struct QueryParams {
  RopeParams rope;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t q_token, q_head, out_token, out_head;  // strides in elements
  const float* weight;
  float eps;
  float inv_d;
  uint32_t h;
  uint32_t groups;          // of heads in a token
};

// kRows heads per eight lanes, one after the other in a token's heads: short
// heads alone would leave too few bytes in flight (d = 192, b = 128, two tokens
// of 128 heads: 6.6 us with one, 5.2 with two, 4.5 with the requests along y).
template <int kUnits, int kRows>
__global__ void __launch_bounds__(kQueryThreads) query_kernel(const __grid_constant__ QueryParams p) {
  const int b = blockIdx.y, l = threadIdx.x % kRowLanes;
  pdl_wait_primary();
  const int32_t L = p.rope.seqlens[b], fresh = p.rope.new_lens ? p.rope.new_lens[b] : p.rope.s;
  const uint32_t group = blockIdx.x * (kQueryThreads / kRowLanes) + threadIdx.x / kRowLanes;  // of the request
  const int j = static_cast<int>(group / p.groups);
  const uint32_t head0 = (group - j * p.groups) * kRows;
  const bool in = j < p.rope.s;
  const int64_t tok = static_cast<int64_t>(b) * p.rope.s + j;
  const __nv_bfloat16* src = p.q + tok * p.q_token + head0 * p.q_head + 8 * l;
  uint4 raw[kRows][kUnits];
  auto load = [&](bool real) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int k = 0; k < kUnits; ++k)
        raw[r][k] = real && head0 + r < p.h ? reinterpret_cast<const uint4*>(src + r * p.q_head)[kRowLanes * k]
                                            : make_uint4(0u, 0u, 0u, 0u);
  };
  // requested before the position is known, unless many tokens may be padding
  if (!p.rope.new_lens) load(in);
  int32_t pos = in ? token_position(L, fresh, p.rope.s, j) : -1;
  const bool turn = p.rope.table != nullptr;
  if (turn && pos >= p.rope.rows) {  // no angles for this position: the rows stay as they were
    if (p.rope.err && l == 0) atomicOr(p.rope.err, MLA_DEVERR_BAD_INDEX);
    pos = -1;
  }
  if (p.rope.new_lens) {
    // whole warps of padding: gone through the rest with nothing to do they took
    // the places of others (5 requests of up to 600 tokens of 64 x 512: 47 us, 40 so)
    if (!__any_sync(0xffffffffu, pos >= 0)) return;
    load(pos >= 0);
  }
  Turn t = {};
  if (turn && pos >= 0) load_turn(t, p.rope.table, pos, l, p.rope.style);
  float inv[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    inv[r] = 1.f;
    if (p.eps > 0.f) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        float x[8];
        unpack8(raw[r][k], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
      }
      inv[r] = 1.f / sqrtf(row_sum(sum) * p.inv_d + p.eps);
    }
  }
  __nv_bfloat16* dst = p.out + tok * p.out_token + head0 * p.out_head + 8 * l;
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const bool turns = turn && k == kUnits - 1;
    if (p.eps > 0.f || turns) {
      float w[8];
      if (p.weight) {
        const float4* at = reinterpret_cast<const float4*>(p.weight) + 2 * (kRowLanes * k + l);
        const float4 w0 = at[0], w1 = at[1];
        w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
        w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float x[8];
        unpack8(raw[r][k], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv[r];
        if (p.weight) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= w[i];
        }
        if (turns) rotate8(x, t, l, p.rope.style);
        raw[r][k] = pack8(x);
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (pos >= 0 && head0 + r < p.h) reinterpret_cast<uint4*>(dst + r * p.out_head)[kRowLanes * k] = raw[r][k];
  }
  pdl_launch_dependents();
}

template <int kUnits, int kRows>
int launch_query(QueryParams p, cudaStream_t stream) {
  p.groups = (p.h + kRows - 1) / kRows;
  constexpr int64_t per_block = kQueryThreads / kRowLanes;
  const int64_t blocks = (static_cast<int64_t>(p.rope.s) * p.groups + per_block - 1) / per_block;
  // a request's tokens along x, requests along y (at most 65535 a launch)
  for (int b = 0; b < p.rope.batch; b += 65535) {
    QueryParams part = p;
    part.rope.seqlens += b;
    if (part.rope.new_lens) part.rope.new_lens += b;
    part.q += static_cast<int64_t>(b) * p.rope.s * p.q_token;
    part.out += static_cast<int64_t>(b) * p.rope.s * p.out_token;
    const int n = p.rope.batch - b < 65535 ? p.rope.batch - b : 65535;
    const int rc = launch_step(query_kernel<kUnits, kRows>, part, blocks, n, kQueryThreads, stream, "query kernel launch");
    if (rc != MLA_OK) return rc;
  }
  return MLA_OK;
}

// Heads of a token, and tokens, may be laid out with gaps but not overlap.
bool heads_apart(int64_t token, int64_t head, int h, int d) {
  if (head < d || token < d || token > kMaxTokenStride) return false;
  return h == 1 || (token - d) / (h - 1) >= head;
}

}  // namespace

}  // namespace mla

using namespace mla;

extern "C" int mla_query_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                   const int32_t* cache_seqlens, const int32_t* new_lens, int batch, int s_q, int h_q,
                                   int d, const float* rope_table, int64_t rope_rows, int rope_style,
                                   const float* norm_weight, float norm_eps, void* out, int64_t out_token_stride,
                                   int64_t out_head_stride, uint32_t* err, cudaStream_t stream) {
  const int rc = check_rope_args(cache_seqlens, batch, s_q, rope_table, rope_rows, rope_style, norm_weight, norm_eps);
  if (rc != MLA_OK) return rc;
  if (!q || !out) return MLA_ERR_NULL;
  if (h_q <= 0 || d < 64 || d > 576 || d % 64 != 0) return MLA_ERR_SHAPE;
  const int64_t rows = static_cast<int64_t>(batch) * s_q * h_q;
  if (rows > (int64_t{1} << 31) - 1) return MLA_ERR_SHAPE;
  if (!heads_apart(q_token_stride, q_head_stride, h_q, d) || !heads_apart(out_token_stride, out_head_stride, h_q, d))
    return MLA_ERR_SHAPE;
  // in place a head's lanes must read what they themselves overwrite
  if (q == out && (q_token_stride != out_token_stride || q_head_stride != out_head_stride)) return MLA_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(out) || (q_token_stride | q_head_stride | out_token_stride | out_head_stride) % 8 != 0)
    return MLA_ERR_ALIGN;

  QueryParams p = {};
  p.rope = {cache_seqlens, new_lens, rope_table, rope_rows, batch, s_q, rope_style, err};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q_token = q_token_stride; p.q_head = q_head_stride;
  p.out_token = out_token_stride; p.out_head = out_head_stride;
  p.weight = norm_weight;
  p.eps = norm_eps;
  p.inv_d = 1.f / static_cast<float>(d);
  p.h = static_cast<uint32_t>(h_q);
  // rotation alone, in place: only the last 64 columns change
  if (norm_eps == 0.f && q == out && q_token_stride == out_token_stride && q_head_stride == out_head_stride) {
    p.q += d - 64;
    p.out += d - 64;
    return launch_query<1, 4>(p, stream);
  }
  switch (d / 64) {
    case 1: return launch_query<1, 4>(p, stream);
    case 2: return launch_query<2, 2>(p, stream);
    case 3: return launch_query<3, 2>(p, stream);
    case 4: return launch_query<4, 1>(p, stream);
    case 5: return launch_query<5, 1>(p, stream);
    case 6: return launch_query<6, 1>(p, stream);
    case 7: return launch_query<7, 1>(p, stream);
    case 8: return launch_query<8, 1>(p, stream);
    default: return launch_query<9, 1>(p, stream);
  }
}
