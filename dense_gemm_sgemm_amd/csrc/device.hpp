// What every C entry point does before it launches: the device check, the
// workspace check, status codes.  Host code only; each library has its own
// copy of the per-device record.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstring>

#include "mi355gemm.h"

namespace mi355gemm {

constexpr int kMaxDevices = 64;

// Returns the current device's CU count, or GEMM_ERR_UNSUPPORTED_DEVICE.
inline int check_device() {
  // Per-device verdict of the gfx950 check: 0 unknown, -1 not supported, else
  // the device's compute-unit count.
  static std::atomic<int> state[kMaxDevices];
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GEMM_ERR_UNSUPPORTED_DEVICE;
  if (dev >= kMaxDevices) return GEMM_ERR_UNSUPPORTED_DEVICE;
  int s = state[dev].load(std::memory_order_acquire);
  if (s == 0) {
    hipDeviceProp_t prop;
    const bool ok = hipGetDeviceProperties(&prop, dev) == hipSuccess &&
                    std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 &&
                    prop.multiProcessorCount > 0;
    s = ok ? prop.multiProcessorCount : -1;
    state[dev].store(s, std::memory_order_release);
  }
  return s > 0 ? s : GEMM_ERR_UNSUPPORTED_DEVICE;
}

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }

inline int to_status(hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

// A caller's workspace: 16-byte aligned and at least `need` bytes (or not
// needed at all).
inline bool workspace_ok(size_t need, const void* ws, unsigned long long bytes) {
  return need == 0 ||
         (ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 15u) == 0 && bytes >= need);
}

}  // namespace mi355gemm
