// Host helpers of the C-ABI front ends, one copy in each library: the
// per-thread error message, the per-device set-up and pointer checks.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "../../include/tgemm.h"

namespace tgemm {
namespace host {
namespace {

thread_local char g_err[1024];

[[maybe_unused]] int fail(int code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

constexpr int kMaxDevices = 64;
std::once_flag g_once[kMaxDevices];
int g_dev_status[kMaxDevices];  // 0 ok, else TGEMM_EHIP
int g_dev_cus[kMaxDevices];     // compute units
char g_dev_msg[kMaxDevices][256];

// more: a further set-up step of the library's own for the device (which is
// current), or nullptr.
void init_device(int dev, hipError_t (*more)(int)) {
  hipDeviceProp_t prop;
  hipError_t e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) {
    g_dev_status[dev] = TGEMM_EHIP;
    snprintf(g_dev_msg[dev], sizeof g_dev_msg[dev], "hipGetDeviceProperties(%d): %s", dev, hipGetErrorString(e));
    return;
  }
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0) {
    g_dev_status[dev] = TGEMM_EHIP;
    snprintf(g_dev_msg[dev], sizeof g_dev_msg[dev], "device %d is %s; this library runs on gfx950 (MI355X) only",
             dev, prop.gcnArchName);
    return;
  }
  g_dev_cus[dev] = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 256;
  if (more && (e = more(dev)) != hipSuccess) {
    g_dev_status[dev] = TGEMM_EHIP;
    snprintf(g_dev_msg[dev], sizeof g_dev_msg[dev], "device %d: address of the scratch array: %s", dev,
             hipGetErrorString(e));
    return;
  }
  g_dev_status[dev] = TGEMM_OK;
}

// Current device, set up once.  Returns TGEMM_OK or TGEMM_EHIP (message set).
[[maybe_unused]] int ensure_device(int *cus, hipError_t (*more)(int)) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(TGEMM_EHIP, "no usable HIP device: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(TGEMM_EHIP, "device index %d out of range", dev);
  std::call_once(g_once[dev], init_device, dev, more);
  if (g_dev_status[dev] != TGEMM_OK) return fail(g_dev_status[dev], "%s", g_dev_msg[dev]);
  if (cus) *cus = g_dev_cus[dev];
  return TGEMM_OK;
}

[[maybe_unused]] bool overlaps(const void *p, uint64_t pn, const void *q, uint64_t qn) {
  if (!p || !q || pn == 0 || qn == 0) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + qn && b < a + pn;
}

[[maybe_unused]] bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }

constexpr uint64_t kOffsetLimit = 0x7fffffffull;  // the kernels use 31-bit buffer offsets

}  // namespace
}  // namespace host
}  // namespace tgemm
