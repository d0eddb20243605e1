// Host helpers shared by the entry points of the C ABI (defined in
// flashmask_api.cu).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstddef>
#include <cstdint>

#include "../../include/flashmask.h"

namespace fm {

// NVTX range around an entry point (visible in a profiler's timeline; a no-op
// when no tool is attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

struct DeviceInfo {
  int sm_count = 0;
  int cc = 0;
  int* status = nullptr;
};

// The calling thread's current device, its SM count and its status word.
int current_device(DeviceInfo* out);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Mask vectors: each pair given whole or not at all, 16-byte aligned.
int check_masks(const int32_t* lts, const int32_t* lte, const int32_t* uts, const int32_t* ute);

// Workspace present, large enough and 256-byte aligned.
int check_ws(const void* ws, size_t have, size_t need);

// FLASHMASK_OK, or FLASHMASK_ERR_CUDA with the text kept for flashmask_strerror.
int cuda_status(cudaError_t e, const char* what);

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Persistent grid of an attention kernel: one CTA per SM, at most one per
// work item, at most the process-wide cap when one is set.
int persistent_grid(int64_t n_items, int sm_count);

// Limit of every bounded device-side wait (flashmask_set_wait_limit_ns).
uint64_t wait_limit_ns();

#define FM_TRY(x)                       \
  do {                                  \
    int _rc = (x);                      \
    if (_rc != FLASHMASK_OK) return _rc; \
  } while (0)
#define FM_CUDA(x) FM_TRY(cuda_status((x), #x))

}  // namespace fm
