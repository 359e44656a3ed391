// tma_host.cuh - host side of TMA: the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace bsa {

// cuTensorMapEncodeTiled, looked up once; null when the driver lacks it.
PFN_cuTensorMapEncodeTiled_v12000 get_encode();

bool device_is_sm100();

}  // namespace bsa
