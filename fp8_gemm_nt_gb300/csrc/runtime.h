// What dg_api.cu keeps per device and per stream, for the other translation units that launch
// kernels: the device's SM count and status word, the stream's workspace, programmatic dependent
// launch, and the record of the last CUDA error.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "dg.h"

namespace dg {

struct LaunchContext {
  int sms = 0;                  // SMs to use (dg_set_num_sms)
  uint32_t* status = nullptr;   // the current device's status word
  bool pdl = false;             // programmatic dependent launch is on
};

// The current device's context; DG_ERR_UNSUPPORTED on a device that is not sm_103.
dg_status launch_context(LaunchContext* out);

// Records `e` for dg_last_cuda_error and returns DG_ERR_CUDA.
dg_status record_cuda_error(cudaError_t e);

// Tensor map of a [rows, cols] weight matrix, E4M3 or packed E2M1 (spread to a byte an element as it is copied),
// copied in boxes of box_rows x 128 columns with the 128-byte swizzle. Maps are cached per host thread. False on
// failure.
bool weight_rows_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows, bool e2m1);

// `bytes` of the stream's workspace, past the arrival counters at its start (kArrivalCounters of them, zero
// between launches: a kernel that counts in them leaves them so). Held until the object goes out of scope, which
// has to be after the launches that use it.
constexpr int kArrivalCounters = 4096;
class StreamWorkspace {
 public:
  StreamWorkspace() = default;
  ~StreamWorkspace();
  StreamWorkspace(const StreamWorkspace&) = delete;
  StreamWorkspace& operator=(const StreamWorkspace&) = delete;
  dg_status acquire(cudaStream_t stream, size_t bytes, void** out);
  int* counters() const { return counters_; }

 private:
  void* lease_ = nullptr;
  int* counters_ = nullptr;
};

// Launches `kernel` on `stream`, as a programmatic dependent of the stream's last kernel if `pdl` (the kernel then
// waits for that one itself, before any access to what it may touch).
template <class... Params, class... Args>
dg_status launch(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, bool pdl, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  return e == cudaSuccess ? DG_OK : record_cuda_error(e);
}

}  // namespace dg
