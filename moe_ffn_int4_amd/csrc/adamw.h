// adamw.h -- launcher of the AdamW step over many tensors (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_int4.h"

namespace moe {

// A launch covers this many tensors: their addresses travel as its arguments, of which a
// kernel has 4 KB, so that a step needs no table in device memory and can be captured.
constexpr int kAdamwTensors = 52;
constexpr int kAdamwBlock = 128;   // elements that share a scale of an 8-bit moment
constexpr int kAdamwChunk = 2048;  // elements of a block of threads
// elements of one call, so that a launch counts its blocks and threads in 32 bits
constexpr int64_t kAdamwMost = int64_t{1} << 34;

hipError_t launch_adamw(const moe_adamw_tensor* tensors, int count, const moe_adamw_hyper& hyper, int bits,
                        hipStream_t stream);

}  // namespace moe
