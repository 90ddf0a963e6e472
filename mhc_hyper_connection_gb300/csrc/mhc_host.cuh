// mhc_host.cuh -- host helpers shared by the API files: the thread's error
// text, device properties, pointer alignment and the tensor-map encoder.
// Defined in mhc_pre_api.cu.
#pragma once

#include <cuda.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mhc_pre.h"

namespace mhc {

struct DeviceInfo {
  bool ok = false;          // an sm_103 part
  int sms = 0;
  size_t max_smem = 0;
  size_t l2_bytes = 0;
};
DeviceInfo device_info(int dev);

// Record the text that mhc_pre_last_error returns, and pass the code on.
mhc_status_t fail(mhc_status_t code, const char* fmt, ...);
void clear_error();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled through the runtime's entry-point lookup; nullptr
// where the driver lacks it.
EncodeTiledFn encode_fn();

}  // namespace mhc
