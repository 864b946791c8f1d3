// pkv_internal.h -- host helpers shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "../../include/pkv.h"

namespace pkv {

// Status for a CUDA runtime error code.
inline int cuda_status(cudaError_t e) {
  return e == cudaSuccess ? PKV_OK : PKV_ECUDA_BASE - static_cast<int>(e);
}

// Device address of the current device's error word (nullptr if it cannot be resolved).
unsigned int* device_error_ptr();

// SM count of the current device (0 on failure).
int sm_count();

// cuTensorMapEncodeTiled from the driver, resolved once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Launches a kernel whose threads all begin with griddep_wait(): its CTAs may take their places
// while the kernel before it ends (programmatic dependent launch), and see all that it wrote. It
// must read it through plain loads: __ldg and const __restrict__ pointers are for data that nothing
// writes while the kernel is resident, and the compiler may move such loads above the wait. It
// lets nothing start early itself. In a row with other short kernels that saves 0.2 to 1 us each
// (append and widening of 64 tokens 4.3 -> 3.4 us, two table calls 9.4 -> 8.8).
template <class... P, class... A>
int launch_waiting(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem,
                   pkv_stream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool valid_block_size(int bs) {
  return bs == 16 || bs == 32 || bs == 64 || bs == 128 || bs == 256;
}

}  // namespace pkv
