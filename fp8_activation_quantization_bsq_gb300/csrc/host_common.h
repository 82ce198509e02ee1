// Host helpers shared by the library's translation units: sizes, argument
// checks, the launch wrapper, and what is looked up once per device.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "bsq.h"

namespace bsq {

inline bool fmt_ok(int32_t f) { return f == BSQ_NVFP4 || f == BSQ_MXFP4 || f == BSQ_MXFP8; }
inline int sf_of(int32_t f) { return f == BSQ_NVFP4 ? 16 : 32; }
inline int atom_cols_of(int32_t f) { return 4 * sf_of(f); }
inline int64_t row_bytes_of(int32_t f, int64_t K) { return f == BSQ_MXFP8 ? K : K / 2; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Launch with programmatic stream serialization (programmatic dependent
// launch): the kernel may start while the previous kernel in the stream
// finishes; each kernel waits (griddepcontrol.wait) before touching memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The current device's SM count and the address of its error word
// (bsq_device_error), which kernels outside bsq.cu get as an argument.
struct HostDevice {
  int index = 0;
  int sm_count = 0;
  unsigned int* error_word = nullptr;
};
bsq_status host_device(HostDevice* out);

// Allow `kernel` `bytes` of dynamic shared memory on device `index` (once per kernel and device).
bsq_status allow_smem(const void* kernel, int bytes, int index);

// cuTensorMapEncodeTiled and cuTensorMapReplaceAddress, or NULL when the driver does not have them.
PFN_cuTensorMapEncodeTiled_v12000 encode_tiled();
PFN_cuTensorMapReplaceAddress_v12000 replace_address();

}  // namespace bsq
