// penalty.hpp -- launcher of the kernel that penalizes logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/libscan.h"

namespace libscan {

hipError_t launch_penalize(const penalty_args_t &a, hipStream_t stream);

}  // namespace libscan
