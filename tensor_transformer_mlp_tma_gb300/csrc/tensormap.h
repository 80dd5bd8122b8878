// The driver's tensor-map encoder, looked up once (tc_gemm.cu); null where the driver has none.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace tpmlp {
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
}
