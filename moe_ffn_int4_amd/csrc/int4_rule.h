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
    k16x64p8,
    k16x256,
    k32x64p4,
    k32x128p2,
    k32x256,
    k48x64p4,
    k64x128,
    k64x256,
    kCount,
};

// What a shape costs, in us: start + round * n + steps * (first + more * (n - 1)), times 1 + narrow
// for the steps of groups of 32, where n tiles fall on a CU and `steps` are the 128-deep
// steps of one part. Fitted to 1100 products of random sizes (1 to 8192 rows, 1 to 128 groups, N 64 to
// 16384, K 128 to 8192) timed with 16 shapes; the times are met to 7 to 16 % (rms), and the shape of the
// least estimate takes 2 % longer than the best of the 16 on average, 14 % and less in 95 of 100, 2.2 times
// in the worst (few rows, dealt unevenly). The twelve were kept one by one for what each saves: of the best five alone
// the least estimate takes 6 % longer.
struct Int4Cost {
    int rows, cols, parts;
    double start, round, first, more, narrow;
};
constexpr Int4Cost kInt4Costs[] = {
    // few strips: 1 x 1024 x 1024 3.6 us (k16x32p8 3.9, k16x64p2 4.6)
    {4, 16, 8, 0.911, 2.640, 0.533, 0.579, 0.054},
    // single rows of many experts: 16 over E = 16, 16384 x 5120 87 (k16x256 84, k16x64p2 103, k32x256 99)
    {4, 128, 2, 3.049, 0.643, 0.717, 0.476, 0.337},
    // few rows of one matrix: 1 x 8192 x 5120 7.7, 16 x 5120 x 8192 10.0 (k16x64p8 13.4, k16x64p2 15.8)
    {16, 32, 8, 1.174, 2.457, 0.798, 0.936, 0.104},
    // 200 over E = 16, 8192 x 5120 91 (k32x64p4 121)
    {16, 64, 2, 2.282, 1.394, 0.474, 0.352, 0.062},
    // 37 x 5120 x 8192 13.7 (k16x32p8 18.0, k32x64p4 18.3, k16x64p2 19.5)
    {16, 64, 8, 1.354, 2.361, 1.249, 1.476, 0.124},
    {16, 256, 1, 2.617, 1.373, 0.717, 0.438, 0.363},
    // 64 x 5120 x 8192 18.9 (k16x64p2 27, k32x128p2 33, k64x128 54)
    {32, 64, 4, 1.106, 2.769, 0.927, 1.046, 0.115},
    // 128 x 5120 x 8192 32.4 (k32x64p4 36, k64x128 54)
    {32, 128, 2, 0.852, 3.233, 0.873, 0.925, 0.150},
    // 1000 over E = 16, 8192 x 5120 152 (k64x128 168, k64x256 157)
    {32, 256, 1, 2.347, 1.209, 1.051, 0.667, 0.300},
    // 100 x 5120 x 8192 25.5 (k32x128p2 32.6, k32x64p4 36.7)
    {48, 64, 4, 0.970, 3.044, 1.183, 1.317, 0.228},
    // 512 x 5120 x 8192 84 (k32x128p2 120, k64x256 89)
    {64, 128, 1, 2.442, 1.083, 0.799, 0.534, 0.471},
    // 4096 x 5120 x 8192 349 (k64x128 387; tiles of 128 x 256, one block a CU, 378)
    {64, 256, 1, 2.248, 1.887, 1.257, 0.977, 0.611},
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
