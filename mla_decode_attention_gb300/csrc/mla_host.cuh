// Host-side helpers that every launch with TMA tensor maps or much shared memory needs.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "mla_decode.h"
#include "mla_internal.h"

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

}  // namespace

}  // namespace mla
