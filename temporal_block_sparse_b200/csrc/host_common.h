// host_common.h -- what the host files of the library share: the per-device set-up, the scratch
// pool and the wait limit, all owned by lite_attn_api.cu.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lite_host {

struct DeviceContext {
  int sms;
  int* status;          // the device status word
  cudaMemPool_t pool;   // the library's stream-ordered scratch pool (null unless asked for)
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  unsigned long long wait_limit_ns;
  int debug_stall;
  int max_ctas;         // 0: no cap
};

// The current device's context; LITE_OK or LITE_ERR_CUDA. with_pool creates the pool on first use.
__attribute__((visibility("hidden"))) int device_context(bool with_pool, DeviceContext* out);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace lite_host
