// Host-side declarations shared by the library's translation units.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mla_decode.h"

namespace mla {

constexpr int kDqk = 576;
constexpr int kDv = 512;
constexpr int kPage = 64;
constexpr int kHeadsPerCta = 64;
constexpr int kMaxSq = 16;

// Supported head counts: 16, 32, 48, 64 (one block) and 128 (two blocks).
inline bool heads_supported(int h) {
  return h == 16 || h == 32 || h == 48 || h == 64 || h == 128;
}
inline int head_blocks(int h) { return (h + kHeadsPerCta - 1) / kHeadsPerCta; }

// Most rows of a packed tensor (all its sequences together), most sequences: what one
// block works on between two signals (a sequence's keys, the search for its next
// item) stays well below the limit of the waits.
constexpr int64_t kMaxPackedRows = int64_t{1} << 25;
constexpr int kMaxSequences = 1 << 16;

inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether rows of `width` elements, `token` apart from token to token and `head` from
// head to head, do not overlap: heads lie within a token, or tokens within a head.
inline bool rows_apart(int64_t tokens, int64_t heads, int64_t token, int64_t head, int64_t width) {
  if (token < 0 || head < 0) return false;
  const bool by_token = (heads == 1 || head >= width) && (tokens == 1 || token >= (heads - 1) * head + width);
  const bool by_head = (tokens == 1 || token >= width) && (heads == 1 || head >= (tokens - 1) * token + width);
  return by_token || by_head;
}

// Records a failed CUDA call for mla_last_error(); returns MLA_ERR_CUDA.
int record_cuda_error(const char* where, cudaError_t e);
// Records a host-side validation failure (no CUDA error).
int record_error(const char* what, int status);

// Host-side range checks of the size arguments shared by the decode entry
// points (the device buffer is never read here; the kernels compare the
// metadata header with the call themselves, see meta_header_matches).
int check_common(int batch, int s_q, int h_q, int num_sm_parts);

// Launches the split combine on `stream`; `pdl` enables programmatic
// dependent launch after the split kernel.
int launch_combine(const void* metadata, int batch, int s_q, int h_q, int num_sm_parts,
                   const void* workspace, const float* attn_sink, void* out, float* lse,
                   cudaStream_t stream, bool pdl);

// Workspace partition: partial O [rows, h, 512] fp32, partial LSE [rows, h]
// fp32, then kWorkspaceCtrlBytes of control words.  Control word 0 holds the
// schedule the last split kernel on this workspace walked (0 = A, 1 = B, -1 =
// metadata rejected); the combine reads it, so the metadata itself is never
// written by a decode call.  Control word 1 is 0 when that schedule left the
// combine nothing to do (schedule B with every sequence non-empty: each one
// written by the split kernel), else 1.
constexpr int64_t kWorkspaceCtrlBytes = 64;
inline int64_t workspace_rows(int batch, int s_q, int num_sm_parts) {
  return static_cast<int64_t>(batch) * s_q + num_sm_parts;
}
inline int32_t* workspace_ctrl(void* workspace, int64_t rows_times_h) {
  return reinterpret_cast<int32_t*>(static_cast<float*>(workspace) + rows_times_h * (kDv + 1));
}
inline const int32_t* workspace_ctrl(const void* workspace, int64_t rows_times_h) {
  return reinterpret_cast<const int32_t*>(static_cast<const float*>(workspace) + rows_times_h * (kDv + 1));
}

}  // namespace mla
