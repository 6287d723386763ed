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
    k32x128p4,
    k32x256,
    k48x64p4,
    k48x256,
    k64x128,
    k64x256,
    kCount,
};

// What a shape costs, in us: start + round * n + steps * (first + more * (n - 1)), times 1 + narrow
// for the steps of groups of 32, where n tiles fall on a CU and `steps` are the 128-deep
// steps of one part. Fitted to 1100 products of random sizes (1 to 8192 rows, 1 to 128 groups, N 64 to
// 16384, K 128 to 8192) timed with 16 shapes; the times are met to 7 to 16 % (rms), and the shape of the
// least estimate takes 2.5 % longer than the best of the 16 on average, 17 % and less in 95 of 100, 1.7 times
// in the worst (few rows, dealt unevenly). The thirteen were kept one by one for what each saves: of the best five alone
// the least estimate takes 7 % longer. Beside each stands a product that it is chosen for, with its time and those of the next.
//
// Where it misses: a group's last tile counts as half empty, and tiles as if a CU had one at a time, so tens of rows an
// expert can go to a neighbouring shape. By the least estimate 500 rows over 16 groups, 8192 x 5120, take tiles of 32 x 256, 89 us (of 48 x
// 256 80); 1000 of 64 x 256, 145 (of 32 x 256 130); 110 over 64, 576 x 7552, of 16 x 64 in eight parts, 32 (in two parts 27).
struct Int4Cost {
    int rows, cols, parts;
    double start, round, first, more, narrow;
};
constexpr Int4Cost kInt4Costs[] = {
    // few strips: 1 x 1024 x 1024 3.8 us (k16x32p8 4.4, k16x64p8 4.7)
    {4, 16, 8, 0.761, 2.725, 0.514, 0.490, 0.090},
    // single rows of many experts: 10 over E = 16, 5248 x 1664 11.6 (k16x256 14.0, k16x64p2 14.4)
    {4, 128, 2, 2.955, 0.661, 0.629, 0.428, 0.297},
    // few rows of one matrix: 1 x 8192 x 5120 7.5 (k16x64p8 9.5), 16 x 5120 x 8192 9.6 (k16x64p8 13.0, k32x64p4 17.3)
    {16, 32, 8, 1.025, 2.484, 0.752, 0.826, 0.159},
    // tens of rows, short reductions: 59 x 2800 x 256 3.6 (k32x64p4 3.9, k16x64p8 4.1)
    {16, 64, 2, 2.116, 1.469, 0.444, 0.311, 0.101},
    // 37 x 5120 x 8192 13.7 (k32x64p4 17.9, k16x32p8 18.4)
    {16, 64, 8, 1.168, 2.468, 1.163, 1.326, 0.171},
    // 16 over E = 16, 16384 x 5120 93 (k32x256 98, k16x64p2 118)
    {16, 256, 1, 2.632, 1.341, 0.599, 0.394, 0.320},
    // 64 x 5120 x 8192 17.9 (k48x64p4 22.6, k16x64p8 25.4)
    {32, 64, 4, 0.903, 2.823, 0.836, 0.936, 0.231},
    // 192 x 5120 x 8192 29.2 (k32x64p4 35.1, k48x64p4 43.3)
    {32, 128, 4, 0.733, 3.357, 1.370, 1.485, 0.276},
    // 2867 over E = 128, 3200 x 1152 59 (k48x256 67, k16x256 76)
    {32, 256, 1, 2.315, 1.225, 0.799, 0.553, 0.259},
    // 100 x 5120 x 8192 23.3 (k32x128p4 27.6, k32x64p4 33.9)
    {48, 64, 4, 0.848, 3.100, 1.086, 1.166, 0.225},
    // 1308 over E = 32, 8880 x 3840 142 (k32x256 174, k64x256 176), 512 x 5120 x 8192 66 (k64x128 73)
    {48, 256, 1, 1.943, 1.842, 0.974, 0.718, 0.262},
    // thousands of rows, few columns: 3012 x 608 x 896 9.0 (k48x256 10.6, k64x256 11.9)
    {64, 128, 1, 2.401, 1.031, 0.778, 0.505, 0.187},
    // 4096 x 5120 x 8192 313 (k48x256 348, k64x128 352)
    {64, 256, 1, 2.190, 1.887, 1.126, 0.894, 0.306},
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
