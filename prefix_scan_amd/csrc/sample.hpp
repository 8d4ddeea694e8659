// sample.hpp -- launcher of the sampling kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/libscan.h"

namespace libscan {

size_t sample_body_bytes(uint64_t rows, uint64_t vocab);
hipError_t launch_sample(const sample_args_t &a, void *body, hipStream_t stream);

}  // namespace libscan
