// gq_host.h -- host helpers shared by the translation units of libgq
// (defined in gq_api.cu; hidden, not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stddef.h>
#include <stdint.h>

#include "gq.h"

namespace gq {

constexpr int kMaxDevices = 64;

int sm_count();                                        // of the current device
bool aligned(const void* p, size_t a);
int64_t packed_row_bytes(int64_t cols, int qbits);
gq_status cuda_status(cudaError_t e);                  // GQ_OK, or GQ_ERR_CUDA with the error recorded
gq_status launch_status();                             // of the launch just made
PFN_cuTensorMapEncodeTiled encode_tiled();             // null if the driver has none

}  // namespace gq
