// The driver's call that describes a tensor to TMA, reached through the runtime (the
// library does not link the driver library itself).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace gdn {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// nullptr where the driver has none (looked for again by the next call).
inline EncodeTiled encode_tiled() {
  static std::atomic<EncodeTiled> known{nullptr};
  if (EncodeTiled f = known.load(std::memory_order_acquire)) return f;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess) {
    cudaGetLastError();                  // clear it
    return nullptr;
  }
  known.store(reinterpret_cast<EncodeTiled>(fn), std::memory_order_release);
  return reinterpret_cast<EncodeTiled>(fn);
}

}  // namespace gdn
