// Host helpers of the C entry points (defined in api.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace skl {

int* status_word();   // the device status word, or null
int check_device();   // STREAMKL_OK on an sm_103a device
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
int l2_head_group(int BH, double bytes_per_head);  // heads whose CTAs interleave (FwdArgs::head_group)

}  // namespace skl
