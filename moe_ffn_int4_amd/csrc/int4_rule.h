// int4_rule.h -- which shape of the kernel of int4.hip computes a product. Host code without
// HIP, so that the rule can be asked on a machine without a GPU.
#pragma once

#include <stdint.h>

#include "matmul_rule.h"

namespace moe {

// rows x columns of a tile, and the parts of its reduction where there are several
enum class Int4Shape {
    k4x16p8,
    k4x128p2,
    k16x32p8,
    k16x64p2,
    k16x64p4,
    k16x256,
    k32x64p4,
    k32x128p2,
    k32x256,
    k64x128,
    k64x256,
    kCount,
};

// What a shape costs, in us: start + round * n + steps * (first + more * (n - 1)), times 1 + narrow
// for the steps of groups of 32, where n tiles fall on a CU and `steps` are the 128-deep
// steps of one part. Fitted to 900 products of random sizes (1 to 8192 rows, 1 to 128 groups, N 64 to
// 16384, K 128 to 8192) timed with 22 shapes; the times are met to 7 to 16 % (rms), and the shape of the
// least estimate takes 3 % longer than the best of the 22 on average, 15 % and less in 95 of 100.
// The eleven were kept one by one for what each saves: with the best two alone 21 %.
struct Int4Cost {
    int rows, cols, parts;
    double start, round, first, more, narrow;
};
constexpr Int4Cost kInt4Costs[] = {
    // few strips: 1 x 1024 x 1024 3.6 us (k16x32p8 3.9, k16x64p2 4.6)
    {4, 16, 8, 0.995, 2.621, 0.506, 0.585, 0.048},
    // single rows of many experts: 16 over E = 16, 16384 x 5120 88 (k16x256 87, k16x64p2 112)
    {4, 128, 2, 2.996, 0.642, 0.727, 0.440, 0.346},
    // few rows of one matrix: 1 x 8192 x 5120 7.7, 16 x 5120 x 8192 10.0 (k16x64p2 15.8)
    {16, 32, 8, 1.278, 2.391, 0.786, 0.945, 0.096},
    // 200 over E = 16, 8192 x 5120 91 (k32x64p4 121)
    {16, 64, 2, 2.247, 1.385, 0.458, 0.346, 0.137},
    // 37 x 5120 x 8192, groups of 32: 17 (k32x64p4 21, k16x64p2 21)
    {16, 64, 4, 1.036, 2.736, 0.754, 0.808, 0.112},
    {16, 256, 1, 2.582, 1.371, 0.725, 0.444, 0.340},
    // 64 x 5120 x 8192 18.9 (k16x64p2 27, k32x128p2 33, k64x128 54)
    {32, 64, 4, 0.860, 2.855, 0.956, 1.039, 0.112},
    // 128 x 5120 x 8192 32.4 (k32x64p4 36, k64x128 54)
    {32, 128, 2, 0.660, 3.349, 0.907, 0.939, 0.113},
    // 1000 over E = 16, 8192 x 5120 152 (k64x128 168, k64x256 157)
    {32, 256, 1, 2.181, 1.290, 1.017, 0.612, 0.355},
    // 512 x 5120 x 8192 84 (k32x128p2 120, k64x256 89)
    {64, 128, 1, 2.348, 1.082, 0.804, 0.517, 0.470},
    // 4096 x 5120 x 8192 349 (k64x128 387; tiles of 128 x 256, one block a CU, 378)
    {64, 256, 1, 1.998, 1.993, 1.290, 0.934, 0.583},
};
static_assert(sizeof(kInt4Costs) / sizeof(Int4Cost) == static_cast<int>(Int4Shape::kCount), "a cost for each shape");

inline Int4Shape choose_int4(int64_t P, int64_t E, int64_t N, int64_t K, int group) {
    int best = 0;
    double least = 0;
    for (int i = 0; i < static_cast<int>(Int4Shape::kCount); ++i) {
        const Int4Cost& c = kInt4Costs[i];
        const int64_t tiles = row_tiles(MatmulSizes{kFwd, P, E, N, K}, c.rows) * ((N + c.cols - 1) / c.cols);
        const double n = static_cast<double>((tiles + 255) / 256);
        const double steps = static_cast<double>((K / 128 + c.parts - 1) / c.parts);
        const double t = c.start + c.round * n + steps * (c.first + c.more * (n - 1)) * (group == 32 ? 1 + c.narrow : 1);
        if (i == 0 || t < least) {
            least = t;
            best = i;
        }
    }
    return static_cast<Int4Shape>(best);
}

}  // namespace moe
