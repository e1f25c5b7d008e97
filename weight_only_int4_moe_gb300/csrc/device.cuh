// What the host sides of all kernels ask of the device and its driver.

#pragma once

#include <cuda.h>

namespace moe {

// SM count of the current device; MOE_ERR_UNSUPPORTED unless it is sm_103.
int device_sms(int *sms);

// The driver's tensor map encoder (NULL if it has none).
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

}  // namespace moe
