// RMS norm of every query head and rotation of its last 64 columns, one pass:
//   y = x * w / sqrt(mean(x^2) + eps)   (when eps > 0; over the head's d columns)
//   y[d-64 .. d) turned by the token's angles, rounded once to bf16.
//
// Bound by memory: every head is read once and written once.  Eight lanes own
// a head and hold all of it in registers (d / 64 units of 16 bytes a lane), so
// the norm's sum is three shuffles and no column is read twice.
#include "mla_rope.cuh"

namespace mla {

namespace {

constexpr int kQueryThreads = 256;

struct QueryParams {
  RopeParams rope;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t q_token, q_head, out_token, out_head;  // strides in elements
  const float* weight;
  float eps;
  float inv_d;
  uint32_t h, rows;
};

template <int kUnits>
__global__ void __launch_bounds__(kQueryThreads) query_kernel(const __grid_constant__ QueryParams p) {
  const uint32_t row = (blockIdx.x * kQueryThreads + threadIdx.x) / kRowLanes;
  const int l = threadIdx.x % kRowLanes;
  const bool in = row < p.rows;
  const uint32_t tok = in ? row / p.h : 0u, head = in ? row - tok * p.h : 0u;
  const int b = static_cast<int>(tok / static_cast<uint32_t>(p.rope.s)), j = static_cast<int>(tok % static_cast<uint32_t>(p.rope.s));
  const uint4* src = reinterpret_cast<const uint4*>(p.q + tok * p.q_token + head * p.q_head) + l;
  uint4 raw[kUnits];  // requested before the position is known
#pragma unroll
  for (int k = 0; k < kUnits; ++k) raw[k] = in ? src[kRowLanes * k] : make_uint4(0u, 0u, 0u, 0u);
  int32_t pos = in ? token_position(p.rope.seqlens, p.rope.new_lens, p.rope.s, b, j) : -1;
  const bool turn = p.rope.table != nullptr;
  if (turn && pos >= p.rope.rows) {  // no angles for this position: the row stays as it was
    if (p.rope.err && l == 0) atomicOr(p.rope.err, MLA_DEVERR_BAD_INDEX);
    pos = -1;
  }
  Turn t = {};
  if (turn && pos >= 0) load_turn(t, p.rope.table, pos, l, p.rope.style);
  float inv = 1.f;
  if (p.eps > 0.f) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      float x[8];
      unpack8(raw[k], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
    }
    inv = 1.f / sqrtf(row_sum(sum) * p.inv_d + p.eps);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out + tok * p.out_token + head * p.out_head) + l;
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if (p.eps > 0.f || (turn && k == kUnits - 1)) {
      float x[8];
      unpack8(raw[k], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv;
      if (p.weight) {
        const float4* w = reinterpret_cast<const float4*>(p.weight) + 2 * (kRowLanes * k + l);
        const float4 w0 = w[0], w1 = w[1];
        x[0] *= w0.x; x[1] *= w0.y; x[2] *= w0.z; x[3] *= w0.w;
        x[4] *= w1.x; x[5] *= w1.y; x[6] *= w1.z; x[7] *= w1.w;
      }
      if (turn && k == kUnits - 1) rotate8(x, t, l, p.rope.style);
      raw[k] = pack8(x);
    }
    if (pos >= 0) dst[kRowLanes * k] = raw[k];
  }
}

template <int kUnits>
int launch_query(const QueryParams& p, cudaStream_t stream) {
  const uint32_t per_block = kQueryThreads / kRowLanes;
  query_kernel<kUnits><<<(p.rows + per_block - 1) / per_block, kQueryThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? MLA_OK : record_cuda_error("query kernel launch", e);
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
  // heads of a token, and tokens, may be laid out with gaps but not overlap
  if (q_head_stride < d || out_head_stride < d || q_token_stride < (h_q - 1) * q_head_stride + d ||
      out_token_stride < (h_q - 1) * out_head_stride + d)
    return MLA_ERR_SHAPE;
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
  p.rows = static_cast<uint32_t>(rows);
  // rotation alone, in place: only the last 64 columns change
  if (norm_eps == 0.f && q == out && q_token_stride == out_token_stride && q_head_stride == out_head_stride) {
    p.q += d - 64;
    p.out += d - 64;
    return launch_query<1>(p, stream);
  }
  switch (d / 64) {
    case 1: return launch_query<1>(p, stream);
    case 2: return launch_query<2>(p, stream);
    case 3: return launch_query<3>(p, stream);
    case 4: return launch_query<4>(p, stream);
    case 5: return launch_query<5>(p, stream);
    case 6: return launch_query<6>(p, stream);
    case 7: return launch_query<7>(p, stream);
    case 8: return launch_query<8>(p, stream);
    default: return launch_query<9>(p, stream);
  }
}
