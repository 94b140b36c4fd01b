// Host-side helpers shared by the C-ABI entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/bsfroute.h"

namespace bsf {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sizes beyond any real problem are refused (BSF_ERR_UNSUPPORTED) before a product of them is
// formed, so no grid or offset computation can wrap: at most 2^31 - 1 rows (tokens, or experts x
// rows) of at most 2^24 elements or bytes each.
constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kMaxRowWidth = int64_t(1) << 24;
inline bool fits_rows(int64_t rows, int64_t width) { return rows <= kMaxRows && width <= kMaxRowWidth; }
// E x N weight rows of width K
inline bool fits_weights(int64_t E, int64_t N, int64_t K) {
  return E <= kMaxRows && N <= kMaxRowWidth && fits_rows(E * N, K);
}

// Status of the launch just enqueued (configuration errors only; the kernel
// itself runs asynchronously).
inline bsf_status launch_status() {
  const cudaError_t err = cudaGetLastError();
  return err == cudaSuccess ? BSF_OK : BSF_ERR_CUDA;
}

// Launch configuration of a programmatic dependent (cudaLaunchAttributeProgrammaticStreamSerialization; an
// ordinary launch if the library is built with BSF_DISABLE_PDL) and, if `cluster` is not 0, of clusters of that many
// CTAs.  The kernel's CTAs may be scheduled while the preceding kernel on `stream` drains, so it must call
// pdl_wait() before its first load from or store to global memory.  (A prefetch into L2 may come earlier: it
// returns nothing, and what the preceding kernel still writes is written in L2.)
struct DependentLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  DependentLaunch(dim3 grid, unsigned block, size_t smem, cudaStream_t stream, unsigned cluster = 0) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    if (cluster != 0) {
      attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      attr[cfg.numAttrs].val.clusterDim.x = cluster;
      attr[cfg.numAttrs].val.clusterDim.y = 1;
      attr[cfg.numAttrs].val.clusterDim.z = 1;
      ++cfg.numAttrs;
    }
#ifndef BSF_DISABLE_PDL
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
#endif
  }
  DependentLaunch(const DependentLaunch&) = delete;        // (cfg points into attr)
  DependentLaunch& operator=(const DependentLaunch&) = delete;
};

// Launch `kernel` as a programmatic dependent.  Returns the launch's configuration status.
template <class... Params, class... Args>
inline bsf_status launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem,
                                   cudaStream_t stream, Args&&... args) {
  DependentLaunch launch(grid, block, smem, stream);
  if (cudaLaunchKernelEx(&launch.cfg, kernel, static_cast<Args&&>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return BSF_ERR_CUDA;
  }
  return launch_status();
}

// Per-device values the library resolves on first use are cached in atomics, so
// first calls from several host threads at once are well defined (each stores
// the same value).  The caches are not invalidated: after cudaDeviceReset() the
// process must not call the library again on that device.

// Number of SMs of the current device (cached per device).
int sm_count();

// Device address of the library's sticky error word on the current device
// (nullptr if it cannot be resolved).
int* device_error_ptr();

}  // namespace bsf
