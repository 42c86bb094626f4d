// host_state.h — per-device host state shared by the library's host files (hstu_attn.cu defines it).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

namespace hstu {

struct DeviceState {
  std::once_flag once;
  cudaError_t init_err = cudaSuccess;
  int num_sms = 0;
  int gemm_clusters = 0;  // resident two-CTA clusters of the two-SM GEMM
  cudaMemPool_t pool = nullptr;
  unsigned* err_word = nullptr;
};

// State of the current device, set up on first use; null if that failed.
DeviceState* device_state();

// The driver's tensor-map encoder; null if the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

}  // namespace hstu
