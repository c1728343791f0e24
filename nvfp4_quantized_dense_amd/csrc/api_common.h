// api_common.h -- what the files of extern "C" entry points share: the error
// text, checks of arguments and of the device.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/nvfp4.h"

namespace nvfp4 {
namespace api {

inline thread_local char g_err[512] = "";

inline int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Largest GEMM dimension accepted: keeps every index of the 32-bit grid
// arithmetic and the 64-bit byte offsets far from overflow.
constexpr int64_t kMaxDim = int64_t(1) << 24;

inline bool dim_ok(int64_t v) { return v >= 0 && v <= kMaxDim; }

// gfx950 check, cached per device.
inline int check_device() {
  static std::mutex mu;
  static int cached[64];
  static bool init = false;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return fail(NVFP4_ERR_HIP, "hipGetDevice failed");
  if (dev < 0 || dev >= 64) return fail(NVFP4_ERR_UNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lock(mu);
  if (!init) {
    for (int& c : cached) c = -1;
    init = true;
  }
  if (cached[dev] < 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
      return fail(NVFP4_ERR_HIP, "hipGetDeviceProperties failed");
    cached[dev] = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 0;
    if (!cached[dev]) {
      fail(NVFP4_ERR_UNSUPPORTED, "device %d is %s; this library runs on gfx950 (MI355X) only", dev,
           prop.gcnArchName);
    }
  }
  if (cached[dev] != 1)
    return fail(NVFP4_ERR_UNSUPPORTED, "device %d is not gfx950 (MI355X); no other path exists", dev);
  return NVFP4_OK;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(NVFP4_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  g_err[0] = '\0';
  return NVFP4_OK;
}

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace api
}  // namespace nvfp4
