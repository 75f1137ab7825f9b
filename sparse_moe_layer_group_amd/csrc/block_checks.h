// Argument checks and workspace layout that the entry points of the operators
// around the expert layer share (block_api.cpp, mx_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "../../include/moe.h"

namespace moe {
namespace checks {

constexpr int64_t kMaxRows = int64_t(1) << 24, kMaxLd = int64_t(1) << 22;
constexpr int32_t kMaxDim = 131072;

#define MOE_TRY(expr)                             \
  do {                                            \
    if ((expr) != hipSuccess) return MOE_ERR_HIP; \
  } while (0)

// the current device is a gfx950 GPU (cached per device)
inline int check_device() {
  static std::atomic<int> state[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return MOE_ERR_HIP;
  if (dev < 0 || dev >= 64) return MOE_ERR_DEVICE;
  int st = state[dev].load(std::memory_order_relaxed);
  if (st == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOE_ERR_HIP;
    st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    state[dev].store(st, std::memory_order_relaxed);
  }
  return st == 1 ? MOE_OK : MOE_ERR_DEVICE;
}

inline int check_dtype(int32_t dt) { return dt == MOE_F32 || dt == MOE_BF16 ? MOE_OK : MOE_ERR_DTYPE; }
inline bool bad_dim(int32_t d) { return d < 1 || d > kMaxDim; }
inline bool bad_rows(int64_t T) { return T < 0 || T > kMaxRows; }
inline bool bad_ld(const void* p, int64_t ld, int64_t cols) { return p != nullptr && (ld < cols || ld >= kMaxLd); }
inline bool bad_ws(const void* ws, size_t have, size_t need) {
  return need > 0 && (ws == nullptr || have < need || (reinterpret_cast<uintptr_t>(ws) & 15) != 0);
}

// consecutive pieces of a workspace, 256 bytes apart
struct Carver {
  char* base;  // NULL: only the total is wanted
  size_t used = 0;
  template <typename P> P* take(size_t bytes) {
    char* p = base == nullptr ? nullptr : base + used;
    used += (bytes + 255) & ~size_t(255);
    return reinterpret_cast<P*>(p);
  }
};
inline int check_format(int32_t f) { return f == MOE_MX_E4M3 || f == MOE_MX_E2M1 ? MOE_OK : MOE_ERR_DTYPE; }
// codes are read 16 bytes at a time, a row's scales 4
inline bool bad_mx(const void* codes, const void* scales) {
  return (reinterpret_cast<uintptr_t>(codes) & 15) != 0 || (reinterpret_cast<uintptr_t>(scales) & 3) != 0;
}

}  // namespace checks
}  // namespace moe
