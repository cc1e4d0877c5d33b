// Attention outputs over several sets of keys joined by their log-sum-exps:
//   lse = ln sum_i e^lse_i,   out = sum_i e^(lse_i - lse) out_i
// (DeepGEMM & FlashMLA article, section 7 merge formula).
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

constexpr int kThreads = 256;

struct Params {
  const void* parts;                             // bf16 or fp32
  int64_t part_stride, token_stride, head_stride; // elements
  const float* lses;
  int64_t lse_part, lse_head, lse_token;
  int n, heads, d;
  int64_t tokens;
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

// kLanes lanes a row, kUnits units of eight columns a lane.
template <bool kF32, int kLanes, int kUnits>
__global__ void __launch_bounds__(kThreads) merge_kernel(const __grid_constant__ Params p) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const int l = threadIdx.x % kLanes;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
  int64_t tok = row / p.heads;
  const int head = static_cast<int>(row - tok * p.heads);
  bool in = tok < p.tokens;
  if (p.rows_from) in = in && tok >= *p.rows_from && tok < *p.rows_to;
  if (!in) tok = 0;
  const float* lses = p.lses + head * p.lse_head + tok * p.lse_token;
  // the weights of up to kLanes parts at a time; first their maximum and sum
  float top = -INFINITY;
  for (int i = l; i < p.n; i += kLanes) {
    const float v = in ? lses[i * p.lse_part] : -INFINITY;
    top = fmaxf(top, v);
  }
  top = group_max<kLanes>(top);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int i = l; i < p.n; i += kLanes) sum += in ? expf(lses[i * p.lse_part] - ref) : 0.f;
  sum = group_sum<kLanes>(sum);
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);  // (NaN stays)
  float acc[kUnits][8] = {};
  const int64_t at = tok * p.token_stride + head * p.head_stride;
  for (int i0 = 0; i0 < p.n; i0 += kLanes) {
    const int mine = i0 + l;
    const float lse_i = in && mine < p.n ? lses[mine * p.lse_part] : -INFINITY;
    const float w_mine = lse_i == -INFINITY ? 0.f : expf(lse_i - ref) * inv;
    const int here = p.n - i0 < kLanes ? p.n - i0 : kLanes;
    constexpr int kAhead = 4;
    for (int j0 = 0; j0 < here; j0 += kAhead) {
      Unit<kF32> u[kAhead][kUnits];
      float w[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        w[j] = __shfl_sync(0xffffffffu, j0 + j < here ? w_mine : 0.f, (j0 + j) % kLanes, kLanes);
        if (j0 + j >= here) w[j] = 0.f;
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
          if (w[j] != 0.f && 8 * (l + kLanes * k) < p.d)
            u[j][k].load(p.parts, (i0 + j0 + j) * p.part_stride + at + 8 * (l + kLanes * k));
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
          if (w[j] != 0.f && 8 * (l + kLanes * k) < p.d) u[j][k].add(w[j], acc[k]);
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
    const int64_t rows = p.tokens * p.heads, per = kThreads / lanes;
    return launch_step(kernel, p, (rows + per - 1) / per, 1, kThreads, stream, "merge kernel launch");
  };
  if (p.d <= 64) return go(merge_kernel<kF32, 8, 1>, 8);
  if (p.d <= 128) return go(merge_kernel<kF32, 16, 1>, 16);
  if (p.d <= 256) return go(merge_kernel<kF32, 32, 1>, 32);
  return go(merge_kernel<kF32, 32, 2>, 32);
}

}  // namespace merge
}  // namespace mla
