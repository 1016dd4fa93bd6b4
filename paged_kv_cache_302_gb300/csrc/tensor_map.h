// tensor_map.h -- TMA tensor maps, encoded by the driver's cuTensorMapEncodeTiled.
#pragma once

#include <cuda.h>

#include "pa_internal.h"

namespace pa {

// dims, box: innermost first; strides (bytes) of every dimension but the innermost.  Out-of-range elements read as
// zeros.
pa_status encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base,
                            const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                            CUtensorMapSwizzle swizzle);

}  // namespace pa
