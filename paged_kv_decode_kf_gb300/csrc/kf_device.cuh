// kf_device.cuh -- host-side facts that the entry points of every source file need.
#pragma once

#include <cuda_runtime.h>

namespace kf {

// Of the current device (set up on first use): its error word and SM count.
cudaError_t device_facts(unsigned int **err, int *sm_count);
// cuTensorMapEncodeTiled, or null if the driver has none.
void *tensor_map_encoder();

}  // namespace kf
