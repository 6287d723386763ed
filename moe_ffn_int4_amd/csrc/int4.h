// int4.h -- launcher of the products with 4-bit weights (internal to the library).
#pragma once

#include "int4_rule.h"
#include "train.h"

namespace moe {

// y[s] = x[s] (scale * code)_e^T, or linear's bias, activation and residual on it. `m` as for a
// product of kFwd (m.b is not used); q and scales in the tiled order of moe_quantize_int4_tiled, group e's
// after N * K / 2 bytes and N * K / group floats each.
struct Int4Args {
    MatmulArgs m;
    const uint8_t* q;
    const float* scales;
};

hipError_t launch_int4(Int4Shape shape, bool linear, int group, const Int4Args& a, hipStream_t stream);

}  // namespace moe
