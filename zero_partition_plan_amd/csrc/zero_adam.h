// Internal interface between the updates: the device step counter's kernel (zero_step.hip), which the
// step over many tensors (zero_adam_tensors.hip) ends with as well.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zero {
namespace step {

// Enqueue the step counter's advance (or its report) after an update.
hipError_t advance_step(int64_t* d_step, const int32_t* d_skip, int32_t* d_status, uint32_t table_len,
                        hipStream_t stream);

}  // namespace step
}  // namespace zero
