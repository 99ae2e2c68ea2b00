// api_common.h -- what the files of the C ABI share: the device check, the wait limit and the
// test hook of the environment (defined in moe_api.cu), pointer checks.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "moe_topk.h"

namespace moe {

struct DeviceInfo {
  int ok = -1;  // -1 unknown, 0 unsupported, 1 sm_103
  int num_sms = 0;
};

// The current device's properties (cached); MOE_ERR_UNSUPPORTED_DEVICE off sm_103.
moe_status_t device_info(DeviceInfo* out);
// MOE_WAIT_TIMEOUT_NS, or the default limit of every in-kernel wait.
uint64_t wait_timeout_ns();
// MOE_TEST_STALL_PRODUCER: 1 makes the GEMM producers issue nothing.
int test_stall_producer();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace moe

#define MOE_CUDA_TRY(expr)                          \
  do {                                              \
    if ((expr) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)
