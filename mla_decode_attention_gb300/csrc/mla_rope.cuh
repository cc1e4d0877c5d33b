// Device code shared by the kernels that take new tokens' rows before the
// attention: token positions, the rotation of 64 columns, 16-byte row units.
//
// Eight lanes own one row.  A row's 8-column units (16 bytes of bf16) are
// dealt out so that lane l holds unit l of every 64-column chunk: a load or
// store instruction moves whole 128-byte segments, the last chunk is the 64
// rotated columns, and a block of 32, 128 or all columns is reduced over 4 or
// 8 neighbouring lanes.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "mla_decode.h"
#include "mla_internal.h"
#include "mla_ptx.cuh"

namespace mla {

constexpr int kRowLanes = 8;

struct RopeParams {
  const int32_t* seqlens;   // [batch] cached tokens, new ones included
  const int32_t* new_lens;  // optional [batch]: new tokens of the request's s slots
  const float* table;       // optional [rows, 64]: 32 cosines, 32 sines of each position
  int64_t rows;
  int batch, s;             // token slots: batch * s
  int style;                // MLA_ROPE_*
  uint32_t* err;
};

// Position of token slot j of a request of length L, n of whose s slots hold new
// tokens, or -1 for padding (slots past those, positions before the first).
__device__ __forceinline__ int32_t token_position(int32_t L, int32_t n, int s, int j) {
  n = n < 0 ? 0 : (n > s ? s : n);
  if (j >= n || L <= 0) return -1;
  const int32_t pos = L - n + j;
  return pos < 0 ? -1 : pos;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Sum over the eight lanes of a row.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Cosines and sines that lane l of a row needs for its eight of the 64 rotated
// columns.  MLA_ROPE_PAIRS: columns (2i, 2i + 1) turn by angle i, so the lane
// holds four whole pairs; MLA_ROPE_HALVES: columns (i, i + 32) turn by angle i,
// so the other half of each of its eight pairs is in lane l ^ 4.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(Turn& t, const float* table, int32_t pos, int l, int style) {
  const float4* row = reinterpret_cast<const float4*>(table + static_cast<int64_t>(pos) * 64);
  const int at = style == MLA_ROPE_PAIRS ? l : 2 * (l & 3);
  const float4 c0 = row[at], s0 = row[8 + at];
  t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w;
  t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w;
  if (style != MLA_ROPE_PAIRS) {
    const float4 c1 = row[at + 1], s1 = row[9 + at];
    t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
    t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
  }
}

// (a, b) -> (a cos - b sin, a sin + b cos) for every pair, in fp32.  Called by
// all lanes of the warp.
__device__ __forceinline__ void rotate8(float (&x)[8], const Turn& t, int l, int style) {
  if (style == MLA_ROPE_PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * t.c[i] - b * t.s[i];
      x[2 * i + 1] = a * t.s[i] + b * t.c[i];
    }
  } else {
    const float sign = l < 4 ? -1.f : 1.f;  // first half: a cos - b sin; second half: b cos + a sin
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, x[i], 4);
      x[i] = x[i] * t.c[i] + sign * (other * t.s[i]);
    }
  }
}

// Launch of a kernel whose blocks may start while the preceding kernel of the
// stream ends; it waits for that kernel (pdl_wait_primary) before it reads or
// writes anything.
template <class Kernel, class Params>
int launch_step(Kernel kernel, const Params& p, int64_t blocks, int blocks_y, int threads, cudaStream_t stream,
                const char* what) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(blocks_y), 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? MLA_OK : record_cuda_error(what, e);
}

// Elements from one token slot to the next that the entry points accept: more
// than the device's memory holds, and 2^24 times it fits 64 bits.
constexpr int64_t kMaxTokenStride = int64_t{1} << 38;

// Host-side checks of the arguments that the two entry points share.
inline int check_rope_args(const void* seqlens, int batch, int s, const float* table, int64_t rows, int style,
                           const float* norm_weight, float norm_eps) {
  if (!seqlens) return MLA_ERR_NULL;
  if (batch <= 0 || s <= 0 || static_cast<int64_t>(batch) * s > (1 << 24)) return MLA_ERR_SHAPE;
  if (table ? rows <= 0 : rows != 0) return MLA_ERR_SHAPE;
  if (style != MLA_ROPE_PAIRS && style != MLA_ROPE_HALVES) return MLA_ERR_UNSUPPORTED;
  if (!(norm_eps >= 0.f) || !(norm_eps < 1e30f) || (norm_weight && norm_eps == 0.f)) return MLA_ERR_SHAPE;
  if (!aligned16(table) || !aligned16(norm_weight)) return MLA_ERR_ALIGN;
  return MLA_OK;
}

}  // namespace mla
