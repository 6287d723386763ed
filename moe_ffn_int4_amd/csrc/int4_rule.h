// int4_rule.h -- which shape of the kernel of int4.hip computes a product. Host code without
// HIP, so that the rule can be asked on a machine without a GPU.
#pragma once

#include <stdint.h>

namespace moe {

enum class Int4Shape {
    kFewWide,   // up to 4 rows, 32 columns, the reduction over 8 parts
    kFew,       // 4 rows, 64 columns, 4 parts
    kRows16,    // 16 rows, 64 columns, 4 parts
    kRows32,    // 32 rows, 64 columns, 4 parts
    kRows64,    // 64 rows, 64 columns, 2 parts
    kTile64,    // tiles of 64 x 128
    kTile128,   // tiles of 128 x 256
};

// Mean rows of the groups that have some, were the rows dealt evenly; strips of 16 columns.
inline Int4Shape choose_int4(int64_t P, int64_t E, int64_t N) {
    const int64_t groups = E < P ? E : P, rows = (P + groups - 1) / groups;
    const int64_t strips = groups * (N / 16);
    if (rows <= 4) return strips <= 1024 ? Int4Shape::kFewWide : Int4Shape::kFew;
    if (rows <= 16) return Int4Shape::kRows16;
    if (rows <= 32) return Int4Shape::kRows32;
    if (rows <= 64) return Int4Shape::kRows64;
    if (rows <= 512) return Int4Shape::kTile64;
    return Int4Shape::kTile128;
}

}  // namespace moe
