// api_util.h -- argument-check helpers shared by the C-ABI sources. Everything
// here has internal linkage: each source keeps its own copy.
#pragma once

#include <hip/hip_runtime.h>
#include <string.h>

#include "../../include/hif4.h"

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// 0 = unknown, 1 = gfx950, 2 = other. Benign race: every writer stores the
// same value for a device.
int g_dev_kind[64];

hif4_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return HIF4_ERR_DEVICE;
  if (dev < 64 && g_dev_kind[dev] != 0) return g_dev_kind[dev] == 1 ? HIF4_OK : HIF4_ERR_DEVICE;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return HIF4_ERR_DEVICE;
  const bool ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < 64) g_dev_kind[dev] = ok ? 1 : 2;
  return ok ? HIF4_OK : HIF4_ERR_DEVICE;
}

hif4_status launched(hipError_t e) { return e == hipSuccess ? HIF4_OK : HIF4_ERR_LAUNCH; }

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace
