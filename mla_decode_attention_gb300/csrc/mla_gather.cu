// Cached tokens read back: rows of several requests from the paged cache, in any of its
// formats, into packed bf16 rows (the keys and values of a prompt's context are
// projected up from them).
//
// Bound by memory.  One warp of a block finds its rows' requests, positions and pages,
// a row a lane; then every thread moves units of 16 columns: 16 codes in and 32 bytes
// out, or 32 bytes in and out, neighbouring threads neighbouring units of a row.
#include "mla_rope.cuh"
#include "mla_splitkv.cuh"

namespace mla {

namespace {

constexpr int kRowsAtOnce = 8;  // rows of a block, times its steps

struct GatherParams {
  const uint8_t* cache;
  int64_t num_pages;
  const int32_t* block_table;
  int64_t bt_stride, bt_width;
  const int32_t* cu;      // [batch + 1]
  const int32_t* starts;  // optional [batch]
  int batch;
  int64_t rows;
  __nv_bfloat16* out;
  int64_t out_row;        // elements from row to row
  int wide;               // rows of out begin on 32 bytes
  uint32_t* err;
};

template <int kFormat>
struct GatherShape {
  static constexpr int kWidth = kFormat == MLA_KV_FP8_528 ? kV41HeadDim : kDqk;
  static constexpr int kUnits = kWidth / 16;
  static constexpr int kThreads = kUnits * kRowsAtOnce;
  static constexpr int kTokenBytes = kFormat == MLA_KV_BF16 ? 2 * kDqk : (kFormat == MLA_KV_FP8_656 ? kFp8TokenBytes : kFp8V41TokenBytes);
};

// A row's source: bytes into the cache; or zeros, or nothing to write.
constexpr int64_t kZeros = -1, kNothing = -2;

__device__ __forceinline__ int64_t row_source(const GatherParams& p, int64_t row, int token_bytes) {
  // the last request that begins at or before the row
  int lo = 0, hi = p.batch;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid + 1] <= row) lo = mid + 1;
    else hi = mid;
  }
  if (lo >= p.batch) return kNothing;
  const int64_t first = p.cu[lo];
  if (row < first) return kNothing;
  const int64_t pos = row - first + (p.starts ? p.starts[lo] : 0);
  const int64_t pg = pos / kPage;
  const int32_t page = pos >= 0 && pg < p.bt_width ? p.block_table[lo * p.bt_stride + pg] : -1;
  if (page < 0 || page >= p.num_pages) {
    if (p.err) atomicOr(p.err, MLA_DEVERR_BAD_PAGE);
    return kZeros;
  }
  return (static_cast<int64_t>(page) * kPage + pos % kPage) * token_bytes;
}

// 32 bytes, a whole sector, by one thread.
__device__ __forceinline__ void st_global_v8(void* to, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x),
               "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// 16 codes and their scale -> 16 bf16 values, each the exact product in fp32 rounded once.
__device__ __forceinline__ void decode16(uint4 codes, float scale, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] & 0xFFFFu)));
    const float2 b = f16x2_to_f32x2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16)));
    o[2 * i] = pack_bf16x2(a.x * scale, a.y * scale);
    o[2 * i + 1] = pack_bf16x2(b.x * scale, b.y * scale);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// kSteps: rows that a thread has on their way at once.  Two for long calls, one for short
// ones, where more blocks count for more (110592 rows of the 656-byte cache: 37 us
// with one, 32 with two; 9189 rows of the 528-byte one 3.4 and 3.8).
template <int kFormat, int kSteps>
__global__ void __launch_bounds__(GatherShape<kFormat>::kThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  using Shape = GatherShape<kFormat>;
  constexpr int kRows = kRowsAtOnce * kSteps;
  __shared__ int64_t src[kRows];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows;
  pdl_launch_dependents();
  pdl_wait_primary();
  if (threadIdx.x < kRows) {
    const int64_t row = row0 + threadIdx.x;
    src[threadIdx.x] = row < p.rows ? row_source(p, row, Shape::kTokenBytes) : kNothing;
  }
  __syncthreads();
  const int unit = threadIdx.x % Shape::kUnits, r0 = threadIdx.x / Shape::kUnits;
  constexpr int kCodeUnits = kDv / 16;
  uint4 a[kSteps], b[kSteps];
  float scale[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t s = src[r0 + kRowsAtOnce * i];
    a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = 0.f;
    if (s < 0) continue;
    const uint8_t* row = p.cache + s;
    if (kFormat == MLA_KV_BF16 || (kFormat == MLA_KV_FP8_656 && unit >= kCodeUnits)) {
      const uint4* at = reinterpret_cast<const uint4*>(kFormat == MLA_KV_BF16 ? row + 32 * unit : row + kFp8RopeOffset + 32 * (unit - kCodeUnits));
      a[i] = at[0];
      b[i] = at[1];
    } else {
      a[i] = reinterpret_cast<const uint4*>(row)[unit];
      if (kFormat == MLA_KV_FP8_656)
        scale[i] = reinterpret_cast<const float*>(row + kFp8ScaleOffset)[unit / 8];
      else
        scale[i] = e8m0_to_f32(row[kV41HeadDim + unit / 2]);
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t s = src[r0 + kRowsAtOnce * i];
    if (s == kNothing) continue;
    if (!(kFormat == MLA_KV_BF16 || (kFormat == MLA_KV_FP8_656 && unit >= kCodeUnits))) decode16(a[i], scale[i], a[i], b[i]);
    uint4* dst = reinterpret_cast<uint4*>(p.out + (row0 + r0 + kRowsAtOnce * i) * p.out_row) + 2 * unit;
    if (p.wide) {  // whole sectors (37.4 us with 16-byte stores, 31.9 so)
      st_global_v8(dst, a[i], b[i]);
    } else {
      dst[0] = a[i];
      dst[1] = b[i];
    }
  }
}

constexpr int64_t kShortRows = 12288;

template <int kFormat>
int launch_gather(const GatherParams& p, cudaStream_t stream) {
  const bool few = p.rows < kShortRows;
  const int per = kRowsAtOnce * (few ? 1 : 2);
  return launch_step(few ? gather_kernel<kFormat, 1> : gather_kernel<kFormat, 2>, p, (p.rows + per - 1) / per, 1,
                     GatherShape<kFormat>::kThreads, stream, "gather kernel launch");
}

}  // namespace

}  // namespace mla

using namespace mla;

extern "C" int mla_gather_kv(const void* kv_cache, int kv_format, int64_t num_pages, const int32_t* block_table,
                             int64_t block_table_stride, int64_t max_pages, const int32_t* cu_seqlens, const int32_t* starts,
                             int batch, int64_t rows, void* out, int64_t out_stride, uint32_t* err, cudaStream_t stream) {
  if (kv_format != MLA_KV_BF16 && kv_format != MLA_KV_FP8_656 && kv_format != MLA_KV_FP8_528) return MLA_ERR_UNSUPPORTED;
  if (batch <= 0 || batch > kMaxSequences || rows < 0 || rows > kMaxPackedRows) return MLA_ERR_SHAPE;
  if (num_pages <= 0 || num_pages > (int64_t{1} << 25) || max_pages <= 0 || (batch > 1 && block_table_stride < max_pages))
    return MLA_ERR_SHAPE;
  if (out_stride < (kv_format == MLA_KV_FP8_528 ? kV41HeadDim : kDqk) || out_stride > kMaxTokenStride) return MLA_ERR_SHAPE;
  if (rows == 0) return MLA_OK;
  if (!kv_cache || !block_table || !cu_seqlens || !out) return MLA_ERR_NULL;
  if (!aligned16(kv_cache) || !aligned16(out) || out_stride % 8 != 0) return MLA_ERR_ALIGN;
  const GatherParams p = {static_cast<const uint8_t*>(kv_cache), num_pages, block_table, block_table_stride, max_pages, cu_seqlens,
                          starts, batch, rows, static_cast<__nv_bfloat16*>(out), out_stride, aligned32(out) && out_stride % 16 == 0, err};
  if (kv_format == MLA_KV_BF16) return launch_gather<MLA_KV_BF16>(p, stream);
  if (kv_format == MLA_KV_FP8_656) return launch_gather<MLA_KV_FP8_656>(p, stream);
  return launch_gather<MLA_KV_FP8_528>(p, stream);
}
