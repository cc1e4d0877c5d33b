// Attention outputs over several sets of keys joined by their log-sum-exps:
//   lse = ln sum_i e^lse_i,   out = sum_i e^(lse_i - lse) out_i.
//
// Bound by memory: n rows in, one out, nothing read twice.  A group of lanes owns a
// row of one token and head, eight columns a lane and step, so a row moves in whole
// lines and its log-sum-exps are weighed by shuffles.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "mla_decode.h"
#include "mla_internal.h"
#include "mla_ptx.cuh"
#include "mla_rope.cuh"

namespace mla {
namespace merge {

constexpr int kThreads = 128;

struct Params {
  const void* parts;                             // bf16 or fp32
  int64_t part_stride, token_stride, head_stride; // elements
  const float* lses;
  int64_t lse_part, lse_head, lse_token;
  int n, heads, d;
  uint32_t tokens;
  const int32_t* rows_from;  // optional: only tokens [*rows_from, *rows_to) are written
  const int32_t* rows_to;
  __nv_bfloat16* out;
  int64_t out_token, out_head;
  float* lse;
  int64_t out_lse_head, out_lse_token;
};

template <int kLanes>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <bool kF32>
struct Unit {
  uint4 a, b;  // eight columns; b: the second four of fp32
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (kF32) {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
      a = s[0];
      b = s[1];
    } else {
      a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    }
  }
  __device__ __forceinline__ void add(float w, float (&acc)[8]) const {
    float x[8];
    if constexpr (kF32) {
      x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
      x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y); x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
    } else {
      unpack8(a, x);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += w * x[i];
  }
};

// Blocks on an SM, as far as registers go: the more rows are on their way the better
// (five states of 2048 x 128 heads x 128: 93 us with 3 blocks of 256 threads, 74 = 5.5 TB/s so;
// 82 with half as many parts in flight and more blocks, 78 with blocks that walk several rows).
template <bool kF32, int kUnits, int kAhead>
constexpr int kBlocks = kUnits * kAhead * (kF32 ? 2 : 1) < 8 || !(kF32 || kUnits == 2) ? 8 : (kF32 && kUnits == 2 ? 6 : 7);

// kLanes lanes a row, kUnits units of eight columns a lane, kAhead parts' units in flight: the
// first are requested before the weights are known.  (A row read for nothing, because its part
// has no key, leaves no trace.  One whose weight is so small that it rounds to 0 is added all the same: what is
// not finite in it belongs to the sum.)
template <bool kF32, int kLanes, int kUnits, int kAhead>
__global__ void __launch_bounds__(kThreads, kBlocks<kF32, kUnits, kAhead>) merge_kernel(const __grid_constant__ Params p) {
  static_assert(kLanes % kAhead == 0, "parts of a step have their weights in one register each");
  pdl_launch_dependents();
  pdl_wait_primary();
  const int l = threadIdx.x % kLanes;
  const uint32_t row = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const uint32_t t = row / p.heads, head = row - t * p.heads;
  bool in = t < p.tokens;
  if (p.rows_from) in = in && static_cast<int32_t>(t) >= *p.rows_from && static_cast<int32_t>(t) < *p.rows_to;
  const int64_t tok = in ? t : 0;
  const int64_t at = tok * p.token_stride + head * p.head_stride + 8 * l;
  Unit<kF32> u[kAhead][kUnits];
  auto request = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int k = 0; k < kUnits; ++k)
        if (in && i0 + j < p.n && 8 * (l + kLanes * k) < p.d) u[j][k].load(p.parts, (i0 + j) * p.part_stride + at + 8 * kLanes * k);
  };
  request(0);
  const float* lses = p.lses + head * p.lse_head + tok * p.lse_token;
  // the maximum and the sum of all, a lane for each kLanes-th
  float top = -INFINITY, first = -INFINITY;
  for (int i = l; i < p.n; i += kLanes) {
    const float v = in ? lses[i * p.lse_part] : -INFINITY;
    if (i == l) first = v;
    top = fmaxf(top, v);
  }
  top = group_max<kLanes>(top);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = expf(first - ref);
  for (int i = l + kLanes; i < p.n; i += kLanes) sum += in ? expf(lses[i * p.lse_part] - ref) : 0.f;
  sum = group_sum<kLanes>(sum);
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);  // (NaN stays)
  float acc[kUnits][8] = {};
  float w_mine = -1.f;  // (no part)
  for (int i0 = 0; i0 < p.n; i0 += kAhead) {
    if (i0 > 0) request(i0);
    if (i0 % kLanes == 0) {  // the next kLanes parts' weights, a lane each
      const float v = i0 == 0 ? first : (in && i0 + l < p.n ? lses[(i0 + l) * p.lse_part] : -INFINITY);
      w_mine = v == -INFINITY ? -1.f : expf(v - ref) * inv;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const float w = __shfl_sync(0xffffffffu, w_mine, i0 % kLanes + j, kLanes);
#pragma unroll
      for (int k = 0; k < kUnits; ++k)
        if (!(w < 0.f) && 8 * (l + kLanes * k) < p.d) u[j][k].add(w, acc[k]);
    }
  }
  __syncwarp();  // every lane has read the log-sum-exps that lane 0 may write over
  if (!in) return;
#pragma unroll
  for (int k = 0; k < kUnits; ++k)
    if (8 * (l + kLanes * k) < p.d)
      *reinterpret_cast<uint4*>(p.out + tok * p.out_token + head * p.out_head + 8 * (l + kLanes * k)) = pack8(acc[k]);
  if (l == 0) p.lse[head * p.out_lse_head + tok * p.out_lse_token] = sum == 0.f ? -INFINITY : ref + logf(sum);
}

template <bool kF32>
int launch_type(const Params& p, cudaStream_t stream) {
  const auto go = [&](auto kernel, int lanes) {
    const int64_t rows = static_cast<int64_t>(p.tokens) * p.heads, per = kThreads / lanes;
    return launch_step(kernel, p, (rows + per - 1) / per, 1, kThreads, stream, "merge kernel launch");
  };
  constexpr int kMore = kF32 ? 4 : 8;
  if (p.d <= 64) return p.n <= 2 ? go(merge_kernel<kF32, 8, 1, 2>, 8) : go(merge_kernel<kF32, 8, 1, kMore>, 8);
  if (p.d <= 128) return p.n <= 2 ? go(merge_kernel<kF32, 16, 1, 2>, 16) : go(merge_kernel<kF32, 16, 1, kMore>, 16);
  if (p.d <= 256) return p.n <= 2 ? go(merge_kernel<kF32, 32, 1, 2>, 32) : go(merge_kernel<kF32, 32, 1, kMore>, 32);
  return p.n <= 2 ? go(merge_kernel<kF32, 32, 2, 2>, 32) : go(merge_kernel<kF32, 32, 2, kMore / 2>, 32);
}

}  // namespace merge
}  // namespace mla
