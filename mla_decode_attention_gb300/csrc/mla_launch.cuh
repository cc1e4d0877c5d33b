// Host-side launch helpers of the decode kernels: TMA tensor maps, kernel
// configuration, the cluster launches.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "mla_decode.h"
#include "mla_internal.h"
#include "mla_splitkv.cuh"
#include "mla_pair.cuh"

namespace mla {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D bf16 row-major tensor [rows, cols] (cols = 576, or 512 for V4.1
// queries) with row stride `stride_bytes`; boxes of [box_rows x 64 columns]
// with 128-byte swizzle.
bool make_rows_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t stride_bytes,
                   uint32_t box_rows, uint64_t cols = kDqk) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), rows};
  const cuuint64_t strides[1] = {stride_bytes};
  const cuuint32_t box[2] = {64u, box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The paged bf16 cache seen as a 4-D tensor [8-token groups][9 chunks][8
// rows][64 columns] (strides: row 1152 bytes, chunk 128 bytes, group 9216
// bytes); boxes of [8 groups][`chunks`][8 rows][64 columns] (one page's
// chunks, starting at the chunk given at load time) with 128-byte swizzle,
// landing as [group][chunk][row][128 bytes].
bool make_quad_map(CUtensorMap* m, const void* base, uint64_t num_pages, uint32_t chunks) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {64u, 8u, static_cast<cuuint64_t>(kDqk / 64), num_pages * (kPage / 8)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(kDqk) * 2u, 128u, static_cast<cuuint64_t>(kDqk) * 2u * 8u};
  const cuuint32_t box[4] = {64u, 8u, chunks, static_cast<cuuint32_t>(kPage / 8)};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D bf16 tensor [rows, cols] whose rows start `stride_bytes` apart; boxes of
// [box_rows x 64 columns] with 128-byte swizzle.
bool make_strided_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                      uint64_t stride_bytes, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), rows};
  const cuuint64_t strides[1] = {stride_bytes};
  const cuuint32_t box[2] = {64u, box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D byte tensor [rows, cols] whose rows start `stride_bytes` apart; boxes of
// [box_rows x box_cols bytes], not swizzled.
bool make_byte_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                   uint64_t stride_bytes, uint32_t box_cols, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {stride_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Lets a kernel have `bytes` of dynamic shared memory on the current device,
// once per device (`done`: a bit per device; past 64 devices, every time).
template <class Kernel>
int allow_shared_memory(Kernel kernel, int bytes, std::atomic<uint64_t>* done, const char* what) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return record_cuda_error(what, e);
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (done->load(std::memory_order_acquire) & bit) return MLA_OK;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return record_cuda_error(what, e);
  done->fetch_or(bit, std::memory_order_release);
  return MLA_OK;
}

template <KvMode kMode, bool kWindow = false>
int launch_split(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const SplitParams& prm,
                 cudaStream_t stream, const CUtensorMap* tm_codes = nullptr,
                 const CUtensorMap* tm_scales = nullptr) {
  static std::atomic<uint64_t> done{0};  // per instantiation
  const int rc = allow_shared_memory(mla_splitkv_kernel<kMode, kWindow>, kWindow ? kSmemBytesWindow : kSmemBytes, &done,
                                     "cudaFuncSetAttribute(split kernel)");
  if (rc != MLA_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(prm.num_parts * prm.n_hblk, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kWindow ? kSmemBytesWindow : kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = prm.n_hblk;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // windowed: the prologue overlaps the previous kernel, whose results it waits for
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kWindow ? 2 : 1;
  // the FP8 code and scale maps are read only by the FP8 instantiation
  const cudaError_t e = cudaLaunchKernelEx(&cfg, mla_splitkv_kernel<kMode, kWindow>, tm_q, tm_kv,
                                           tm_codes ? *tm_codes : tm_kv,
                                           tm_scales ? *tm_scales : tm_kv, prm);
  return e == cudaSuccess ? MLA_OK : record_cuda_error("split kernel launch", e);
}

// The query rows [n_seq * 128, 576] seen as [9 chunks][rows][64 columns]
// (chunk stride 128 bytes); boxes of [2 chunks x 128 rows x 64 columns] (a
// quarter of the latent part of one token's rows, 32 KB) with 128-byte swizzle.
bool make_q_latent_map(CUtensorMap* m, const void* q, uint64_t rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {64u, rows, static_cast<cuuint64_t>(kDqk / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kDqk) * 2u, 128u};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(pair::kRows), 2u};  // two chunks per box
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// tm_qa, tm_qb: the group-interleaved maps of the paged cache (chunks 0..3,
// 4..6 of a page); the sparse kernel does not read them.  The kernel loads the
// part's first query rows with the two query maps made here.
template <bool kSparse, bool kWindow = false>
int launch_pair(const CUtensorMap& tm_kv, const CUtensorMap& tm_qa, const CUtensorMap& tm_qb,
                const SplitParams& prm, cudaStream_t stream) {
  CUtensorMap tm_ql, tm_qr;
  const uint64_t q_rows = static_cast<uint64_t>(prm.batch) * prm.s_q * prm.h;
  if (!make_q_latent_map(&tm_ql, prm.q, q_rows) || !make_rows_map(&tm_qr, prm.q, q_rows, kDqk * 2, pair::kRows))
    return record_error("cuTensorMapEncodeTiled failed for the query rows", MLA_ERR_CUDA);
  static std::atomic<uint64_t> done{0};  // per instantiation
  const int rc = allow_shared_memory(pair::mla_pair_kernel<kSparse, kWindow>,
                                     kWindow ? pair::kSmemBytesWindow : pair::kSmemBytes, &done,
                                     "cudaFuncSetAttribute(pair kernel)");
  if (rc != MLA_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(prm.num_parts * 2, 1, 1);
  cfg.blockDim = dim3(kSparse ? pair::kThreadsSparse : pair::kThreads, 1, 1);
  cfg.dynamicSmemBytes = kWindow ? pair::kSmemBytesWindow : pair::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // the kernel's prologue overlaps the previous kernel (e.g. the schedule);
  // it waits for that kernel's results before reading any input
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, pair::mla_pair_kernel<kSparse, kWindow>, tm_kv, tm_qa, tm_qb, tm_ql, tm_qr, prm);
  return e == cudaSuccess ? MLA_OK : record_cuda_error("pair kernel launch", e);
}

// The tensor maps of a paged call (the cache at `kv_cache`, the query rows and
// sizes of `prm`), the page groups of the two-SM kernel when `quads`; the ones
// that the format does not use are not set.
struct CacheMaps {
  CUtensorMap q, kv, codes, scales, quad4, quad3;
};
int make_cache_maps(CacheMaps* m, const SplitParams& prm, const void* kv_cache, int kv_format, bool quads) {
  const uint64_t tokens = static_cast<uint64_t>(prm.num_pages) * kPage;
  if (!make_rows_map(&m->q, prm.q, static_cast<uint64_t>(prm.batch) * prm.s_q * prm.h, prm.d_qk * 2, prm.rows, prm.d_qk))
    return record_error("cuTensorMapEncodeTiled failed for q", MLA_ERR_CUDA);
  if (kv_format == MLA_KV_FP8_528) {
    // the 512 e4m3 codes (boxes of 64 tokens x 64 codes) and the 16 e8m0
    // scales at byte 512 (boxes of 64 tokens x 16 bytes) of every 528-byte
    // token; no bf16 part (kv is not read)
    if (!make_byte_map(&m->codes, kv_cache, tokens, kV41HeadDim, kFp8V41TokenBytes, 64, kPage) ||
        !make_byte_map(&m->scales, static_cast<const uint8_t*>(kv_cache) + kV41HeadDim, tokens, 16,
                       kFp8V41TokenBytes, 16, kPage))
      return record_error("cuTensorMapEncodeTiled failed for the V4.1 FP8 codes or scales", MLA_ERR_CUDA);
    m->kv = m->codes;
  } else if (kv_format == MLA_KV_FP8_656) {
    // the bf16 RoPE tail of every 656-byte token: 64 columns at byte 528,
    // row stride 656 bytes (both multiples of 16)
    const void* rope = static_cast<const uint8_t*>(kv_cache) + kFp8RopeOffset;
    if (!make_strided_map(&m->kv, rope, tokens, 64, kFp8TokenBytes, kPage))
      return record_error("cuTensorMapEncodeTiled failed for the FP8 RoPE columns", MLA_ERR_CUDA);
    // the 512 e4m3 codes (boxes of 64 tokens x 64 codes) and the 16 scale
    // bytes at byte 512 (boxes of 64 tokens x 16 bytes) of every token
    if (!make_byte_map(&m->codes, kv_cache, tokens, kFp8ScaleOffset, kFp8TokenBytes, 64, kPage) ||
        !make_byte_map(&m->scales, static_cast<const uint8_t*>(kv_cache) + kFp8ScaleOffset, tokens, 16,
                       kFp8TokenBytes, 16, kPage))
      return record_error("cuTensorMapEncodeTiled failed for the FP8 codes or scales", MLA_ERR_CUDA);
  } else {
    if (!make_rows_map(&m->kv, kv_cache, tokens, kDqk * 2, kPage))
      return record_error("cuTensorMapEncodeTiled failed for kv_cache", MLA_ERR_CUDA);
    if (quads && (!make_quad_map(&m->quad4, kv_cache, static_cast<uint64_t>(prm.num_pages), 4) ||
                                 !make_quad_map(&m->quad3, kv_cache, static_cast<uint64_t>(prm.num_pages), 3)))
      return record_error("cuTensorMapEncodeTiled failed for the kv_cache page groups", MLA_ERR_CUDA);
  }
  return MLA_OK;
}

}  // namespace

}  // namespace mla
