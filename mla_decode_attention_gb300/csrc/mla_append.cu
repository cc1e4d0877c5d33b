// New tokens' latent rows into the paged cache: RMS norm of the 512 latent
// columns, rotation of the 64 position columns, encoding in the cache's format
// and the write to the token's page slot, one pass.
//
// Bound by memory for prompts (a row is read once and written once) and by
// latency for a decode step.  Eight lanes own a token and hold its row in
// registers (nine units of 16 bytes a lane), so the norm and the FP8 scales are
// shuffles among neighbouring lanes.  65536 rows: bf16 cache 28 us = 6.0 TB/s (88
// % of the copy rate); 656-byte cache 37.5 us (53 %) and 528-byte cache 27 us (66
// %).  There 28 % (95 registers a thread) and 39 % of the warps are resident, too
// few for one block's loads to overlap another's encoding; the arithmetic itself is
// not the bound (quotients by the reciprocal, with a division only next to a border
// between two codes: 36.6 of then 37.9 us; 64 registers a thread: 34.8, but 5.6
// instead of 5.0 for a decode step; neither kept).  A decode step takes 3 to 5 us
// whatever its rows: launch, then lengths, page entry, row, one after the other.
#include "mla_rope.cuh"
#include "mla_splitkv.cuh"

namespace mla {

namespace {

constexpr int kAppendThreads = 128;

struct AppendParams {
  RopeParams rope;
  const __nv_bfloat16* x;
  int64_t x_token;          // elements from one token slot to the next
  const float* weight;
  float eps;
  uint8_t* cache;
  int64_t num_pages;
  const int32_t* block_table;
  int64_t bt_stride, bt_width;  // from one row to the next; entries of a row
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ float abs_max8(const float (&x)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return m;
}

// Biased exponent of the smallest power of two at or above ratio (>= 0), at
// least 2^-127; 127 (2^0) for zero.
__device__ __forceinline__ uint32_t e8m0_at_or_above(float ratio) {
  const uint32_t bits = __float_as_uint(ratio);
  const uint32_t e = bits >> 23, m = bits & 0x7FFFFFu;
  if (bits == 0u) return 127u;
  if (e == 0u) return m > 0x400000u ? 1u : 0u;  // subnormal: above 2^-127 or not
  return e + (m != 0u ? 1u : 0u);
}

// kFormat: MLA_KV_*.
template <int kFormat>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kWidth = kFormat == MLA_KV_FP8_528 ? kV41HeadDim : kDqk;
  constexpr int kUnits = kWidth / 64;
  constexpr int kTokenBytes = kFormat == MLA_KV_BF16 ? 2 * kDqk : (kFormat == MLA_KV_FP8_656 ? kFp8TokenBytes : kFp8V41TokenBytes);
  const int tok = (blockIdx.x * kAppendThreads + threadIdx.x) / kRowLanes;
  const int l = threadIdx.x % kRowLanes;
  const bool in = tok < p.rope.batch * p.rope.s;
  const int b = in ? tok / p.rope.s : 0, j = in ? tok - b * p.rope.s : 0;
  const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(tok) * p.x_token) + l;
  uint4 raw[kUnits];
  auto load = [&](bool real) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) raw[k] = real ? src[kRowLanes * k] : make_uint4(0u, 0u, 0u, 0u);
  };
  pdl_wait_primary();
  // requested before the position is known, unless many tokens may be padding
  if (!p.rope.new_lens) load(in);
  int32_t pos = in ? token_position(p.rope.seqlens[b], p.rope.new_lens ? p.rope.new_lens[b] : p.rope.s, p.rope.s, j) : -1;
  const bool turn = p.rope.table != nullptr;
  int64_t slot = 0;
  if (pos >= 0) {
    const int64_t pg = pos / kPage;
    const int32_t page = pg < p.bt_width ? p.block_table[b * p.bt_stride + pg] : -1;
    uint32_t bad = 0u;
    if (page < 0 || page >= p.num_pages) bad |= MLA_DEVERR_BAD_PAGE;
    if (turn && pos >= p.rope.rows) bad |= MLA_DEVERR_BAD_INDEX;
    slot = static_cast<int64_t>(page) * kPage + pos % kPage;
    if (bad) {  // nothing is written for this token
      if (p.rope.err && l == 0) atomicOr(p.rope.err, bad);
      pos = -1;
    }
  }
  if (p.rope.new_lens) {
    // whole warps of padding take no further part (16 requests of up to 4096
    // tokens into the 528-byte cache: 24 us with them, 18 so)
    if (!__any_sync(0xffffffffu, pos >= 0)) return;
    load(pos >= 0);
  }
  Turn t = {};
  if (turn && pos >= 0) load_turn(t, p.rope.table, pos, l, p.rope.style);
  float inv = 1.f;
  if (p.eps > 0.f) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kDv / 64; ++k) {
      float x[8];
      unpack8(raw[k], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
    }
    inv = 1.f / sqrtf(row_sum(sum) * (1.f / kDv) + p.eps);
  }
  // columns 64 k + 8 l .. + 7 of the row that is cached
  auto unit = [&](int k, float (&x)[8]) {
    unpack8(raw[k], x);
    if (k < kDv / 64) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv;
      if (p.weight) {
        const float4* w = reinterpret_cast<const float4*>(p.weight) + 2 * (kRowLanes * k + l);
        const float4 w0 = w[0], w1 = w[1];
        x[0] *= w0.x; x[1] *= w0.y; x[2] *= w0.z; x[3] *= w0.w;
        x[4] *= w1.x; x[5] *= w1.y; x[6] *= w1.z; x[7] *= w1.w;
      }
    }
    if (turn && k == kUnits - 1) rotate8(x, t, l, p.rope.style);
  };
  uint8_t* dst = p.cache + slot * kTokenBytes;
  if constexpr (kFormat == MLA_KV_BF16) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      float x[8];
      unit(k, x);
      if (pos >= 0) reinterpret_cast<uint4*>(dst)[kRowLanes * k + l] = pack8(x);
    }
  } else if constexpr (kFormat == MLA_KV_FP8_656) {
    float4 scales;
#pragma unroll
    for (int tile = 0; tile < 4; ++tile) {  // 128 columns: two units a lane
      float x[8], y[8];
      unit(2 * tile, x);
      unit(2 * tile + 1, y);
      float m = fmaxf(abs_max8(x), abs_max8(y));
#pragma unroll
      for (int o = 1; o < kRowLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      // (at least the least float: a quotient that rounds to 0 would make NaN of 0 / 0)
      const float sc = m > 0.f ? fmaxf(__fdiv_rn(m, 448.f), __uint_as_float(1u)) : 1.f;
      (tile == 0 ? scales.x : tile == 1 ? scales.y : tile == 2 ? scales.z : scales.w) = sc;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = __fdiv_rn(x[i], sc);
        y[i] = __fdiv_rn(y[i], sc);
      }
      if (pos >= 0) {
        uint2* codes = reinterpret_cast<uint2*>(dst + 128 * tile) + l;
        codes[0] = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
        codes[kRowLanes] = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
      }
    }
    float x[8];
    unit(kUnits - 1, x);
    if (pos >= 0) {
      if (l == 0) *reinterpret_cast<float4*>(dst + kFp8ScaleOffset) = scales;
      reinterpret_cast<uint4*>(dst + kFp8RopeOffset)[l] = pack8(x);
    }
  } else {
    uint32_t codes8[4] = {0u, 0u, 0u, 0u};  // the 16 scale codes, two a chunk
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {  // two blocks of 32 columns, four lanes each
      float x[8];
      unit(k, x);
      float m = abs_max8(x);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t e = e8m0_at_or_above(__fdiv_rn(m, 448.f));
      const uint32_t other = __shfl_xor_sync(0xffffffffu, e, 4);
      codes8[k >> 1] |= ((l < 4 ? e : other) | (l < 4 ? other : e) << 8) << (16 * (k & 1));
      // 1 / 2^(e - 127) = 2^(127 - e): exact, a subnormal only past e = 253
      const float up = e < 254u ? __uint_as_float((254u - e) << 23) : __uint_as_float(0x00400000u);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= up;
      if (pos >= 0)
        reinterpret_cast<uint2*>(dst)[kRowLanes * k + l] = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
    }
    if (pos >= 0 && l == 0) *reinterpret_cast<uint4*>(dst + kV41HeadDim) = make_uint4(codes8[0], codes8[1], codes8[2], codes8[3]);
  }
  pdl_launch_dependents();
}

}  // namespace

}  // namespace mla

using namespace mla;

extern "C" int mla_append_kv(const void* kv_new, int64_t token_stride, const int32_t* cache_seqlens,
                             const int32_t* new_lens, int batch, int s_new, const float* rope_table, int64_t rope_rows,
                             int rope_style, const float* norm_weight, float norm_eps, void* kv_cache, int kv_format,
                             int64_t num_pages, const int32_t* block_table, int64_t block_table_stride,
                             int64_t max_pages, uint32_t* err,
                             cudaStream_t stream) {
  const int rc = check_rope_args(cache_seqlens, batch, s_new, rope_table, rope_rows, rope_style, norm_weight, norm_eps);
  if (rc != MLA_OK) return rc;
  if (!kv_new || !kv_cache || !block_table) return MLA_ERR_NULL;
  if (kv_format != MLA_KV_BF16 && kv_format != MLA_KV_FP8_656 && kv_format != MLA_KV_FP8_528)
    return MLA_ERR_UNSUPPORTED;
  if (num_pages <= 0 || num_pages > (int64_t{1} << 25) || max_pages <= 0 ||
      (batch > 1 && block_table_stride < max_pages))
    return MLA_ERR_SHAPE;
  if (token_stride < (kv_format == MLA_KV_FP8_528 ? kV41HeadDim : kDqk) || token_stride > kMaxTokenStride)
    return MLA_ERR_SHAPE;
  if (!aligned16(kv_new) || !aligned16(kv_cache) || token_stride % 8 != 0) return MLA_ERR_ALIGN;

  AppendParams p = {};
  p.rope = {cache_seqlens, new_lens, rope_table, rope_rows, batch, s_new, rope_style, err};
  p.x = static_cast<const __nv_bfloat16*>(kv_new);
  p.x_token = token_stride;
  p.weight = norm_weight;
  p.eps = norm_eps;
  p.cache = static_cast<uint8_t*>(kv_cache);
  p.num_pages = num_pages;
  p.block_table = block_table;
  p.bt_stride = block_table_stride;
  p.bt_width = max_pages;
  const int per_block = kAppendThreads / kRowLanes;
  const int blocks = (batch * s_new + per_block - 1) / per_block;
  const char* what = "append kernel launch";
  if (kv_format == MLA_KV_BF16) return launch_step(append_kernel<MLA_KV_BF16>, p, blocks, 1, kAppendThreads, stream, what);
  if (kv_format == MLA_KV_FP8_656) return launch_step(append_kernel<MLA_KV_FP8_656>, p, blocks, 1, kAppendThreads, stream, what);
  return launch_step(append_kernel<MLA_KV_FP8_528>, p, blocks, 1, kAppendThreads, stream, what);
}
