// pa_launch.h -- host-side facts that launches share: the current device and the
// driver's tensor-map encoder.
#pragma once

#include <cuda.h>

#include "../../include/pa.h"

namespace pa {

struct DeviceInfo { int sms = 0; int max_smem = 0; };
bool device_info(DeviceInfo& info);           // of the current device, kept per device

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();                    // null without a driver
CUtensorMapDataType tmap_type(pa_dtype d);

}  // namespace pa
