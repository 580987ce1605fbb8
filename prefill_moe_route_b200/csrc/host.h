// host.h -- host helpers shared by the C ABI's source files (defined in api.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace moe {

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Records the text moe_last_error returns and passes `code` on.
int fail(int code, const char* what, cudaError_t e = cudaSuccess);

// Tiled tensor map with the 128-byte swizzle; false if the driver rejects it.
bool make_map(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const uint64_t* dims,
              const uint64_t* strides_bytes, const uint32_t* box);

int sm_count(int dev);
uint64_t wait_timeout_ns();   // MOE_WAIT_TIMEOUT_MS
int take_withhold();          // MOE_TEST_WITHHOLD_FLAG: 1 while calls are left that withhold a flag

// Device of the stream, checked against every non-null pointer; <0 is an error code.
int resolve_device(void* stream, const void* const* ptrs, int n);

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

}  // namespace moe
