// tma_host.cuh - host side of TMA: the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace bsa {

// cuTensorMapEncodeTiled, looked up once; null when the driver lacks it.
PFN_cuTensorMapEncodeTiled_v12000 get_encode();

// Map over an 8-bit cache's e4m3 tiles: [rows, D], a 128-row tile per box,
// swizzled over its row (128 bytes, or 64 for D = 64).
bool make_map8(CUtensorMap* m, const void* base, long long rows, int D);

bool device_is_sm100();

}  // namespace bsa
