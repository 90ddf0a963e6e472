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

// Bytes of one tensor of a call (p NULL: not given).
struct Span {
  const char* name;
  const void* p;
  size_t bytes;
};
// MHC_ERR_PARAM_INVALID if an output shares bytes with an input or with another
// output: kernels read inputs while they write outputs.
template <int NO, int NI>
mhc_status_t check_apart(const Span (&outs)[NO], const Span (&ins)[NI]) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && (x < y ? y - x < a.bytes : x - y < b.bytes);
  };
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (meet(outs[o], ins[i])) return fail(MHC_ERR_PARAM_INVALID, "%s overlaps %s", outs[o].name, ins[i].name);
    for (int i = 0; i < o; ++i)
      if (meet(outs[o], outs[i])) return fail(MHC_ERR_PARAM_INVALID, "%s overlaps %s", outs[o].name, outs[i].name);
  }
  return MHC_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled through the runtime's entry-point lookup; nullptr
// where the driver lacks it.
EncodeTiledFn encode_fn();

}  // namespace mhc
