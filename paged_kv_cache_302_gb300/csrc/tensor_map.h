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

// One box is the chunk of one (block, head) of a quantised cache: D bytes, 2 B rows; third coordinate block * H_kv +
// head (NB * H_kv is past the tensor).  Swizzled by row length: 128 bytes (D = 128) or 64 (D = 64).
pa_status quant_tensor_map(CUtensorMap* m, const void* qpool, int NB, int H_kv, int B, int D);

}  // namespace pa
