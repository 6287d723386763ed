// matmul_rule.h -- which of the kernels of matmul.h computes a product. Host code without
// HIP, so that the rule can be asked on a machine without a GPU.
#pragma once

#include <math.h>
#include <stdint.h>

namespace moe {

// products of matmul.h
constexpr int kFwd = 0;
constexpr int kDx = 1;
constexpr int kDw = 2;

struct MatmulSizes {
    int mode;  // kFwd, kDx, kDw
    int64_t P, E, N, K;
};

enum class MatmulKernel {
    kStream,       // matmul_stream.hip
    kSplit32,      // matmul_split.hip
    kTile64Parts,  // matmul_tile.hip: tiles of 64, the reduction in three parts
    kTile64,       // tiles of 64 over four stages
    kTile128Deep,  // tiles of 128 over four stages
    kTile128,      // tiles of 128 over two stages
    kTile256,      // matmul256.hip
};

// Row tiles of T, an estimate where the host does not know the group sizes: each group's
// last one is half empty, and a group shorter than a tile has a whole one. Of E groups as
// many have rows as do when each row falls into any of them alike.
inline int64_t row_tiles(const MatmulSizes& a, int64_t T) {
    const int64_t groups = a.E < a.P ? a.E : a.P;
    if (groups == 1) return (a.P + T - 1) / T;
    const int64_t half = a.P / T + (groups + 1) / 2;
    const double E = static_cast<double>(a.E);
    const int64_t filled = llround(E * (1.0 - pow(1.0 - 1.0 / E, static_cast<double>(a.P))));
    return half > filled ? half : filled;
}

inline int64_t tiles(const MatmulSizes& a, int64_t T) {
    auto up = [T](int64_t v) { return (v + T - 1) / T; };
    if (a.mode == kDw) return a.E * up(a.N) * up(a.K);
    return row_tiles(a, T) * up(a.mode == kFwd ? a.N : a.K);
}

// The kernel for a product. What decides is how many tiles there are for the chip's
// 256 CUs and how long the reduction is (of weight gradients: a group's mean). In us,
// rows x N x K, dense unless E experts are named:
//   * y = x W^T of few rows (up to 16, or 4 an expert): the streaming kernel, if it has up to
//     768 blocks or the reduction is 1024 or more. 16 rows over E = 16, 16384 x 5120: 306 against
//     424 in tiles of 64; but 72 over E = 128, 9408 x 104: 112, in tiles of 128 over two
//     stages 42. Of any rows in up to 128 of its blocks: 46 x 128 x 7856 7.5, in tiles of 32 10.7.
//   * up to 256 tiles of 32 and a reduction of 512 or more: those, split over eight waves.
//     dx of 3 rows, 8704 x 136: 12.1 against 27.1 in tiles of 64, split; 171 x 2984 x 96, dx: 7.8
//     (13.8); dW of 7195 x 160 x 80: 11.3 (25.0); 144 x 904 x 5240 (145): 10.7 (20.3, streaming
//     19.2); 17 x 16384 x 5120, dx (160): 46.8 (50.6); dx of 12 rows over E = 4, 11928 x 3336
//     (about 420): 83.5 (62.3); of 48 rows over E = 128, 8896 x 232 (about 320): 54.6 (37.0).
//   * y = x W^T of up to 768 streaming blocks: those. 300 rows over E = 40, 264 x 504 (about
//     680): 6.0 against 6.7 in tiles of 64; 496 x 120 x 504 (248): 6.2 (6.4).
//   * up to 256 tiles of 64 and a reduction of 768 or more: those, split in three. 100 x
//     4096 x 4096 (128 tiles): 16.1 against 23.5 not split, 18.4 split in two; 256 x 4096 x
//     4096 (256): 21.6 (24.5); dx of 48 rows over E = 128, 8896 x 232 (about 160): 37.0 (52.9);
//     of 640 rows over E = 128, 1024 x 136 (about 380): 14.5 (11.6); 256 x 8192 x 5120 (512):
//     54.1 (51.6); 300 rows over E = 16, 512 x 1024, dx, 512 long: 7.6 (6.7).
//   * up to 512 tiles of 64: those. 256 x 8192 x 5120 (512 tiles): 52 (tiles of 128: 63, of
//     256: 89); 512 x 8192 x 5120 (1024): 92 (66, 86).
//   * up to 256 tiles of 128 and a reduction of 512 or more: those, one block a CU, over four
//     stages (three steps ahead). 512 x 8192 x 5120 (256): 66, with two stages and two
//     blocks a CU 81; 1024 x 8192 x 5120 (512): 124 against 92 in tiles of 256; 161 rows over E =
//     8, 240 x 6208, dx: 13.6, with two stages 9.3.
//   * reductions below 512 or groups of fewer than 128 rows, whose time is the start and
//     the stores: tiles of 128 over two stages, two blocks a CU. 885 x 8248 x 504: 17
//     (tiles of 256: 24); 2312 rows over E = 128, 1192 x 1008, dx: 59 (83); dW of 20 rows in
//     each of E = 128, 1000 x 712: 44 (49); 8946 rows over E = 2, 11000 x 728: 205 (177);
//     dW of 512 rows in each of E = 16, 5120 x 8192: 834 (770).
//   * else tiles of 256. 1024 x 5120 x 8192 (80): 115 (128: 132).
// Over 2700 products of random sizes this takes 2 % longer than the best kernel for each. With a
// group shorter than a tile counted as half a tile, 45 drawn products of groups for which the
// rule then takes another kernel took 14 % longer.
inline MatmulKernel choose_matmul(const MatmulSizes& a) {
    const int64_t red = a.mode == kFwd ? a.K : a.mode == kDx ? a.N : a.P / a.E;
    const bool few = a.P <= 16 || a.P <= 4 * a.E;
    int64_t strips = 0;  // blocks of the streaming kernel
    if (a.mode == kFwd) {
        strips = row_tiles(a, a.P <= 4 * a.E ? 4 : 16) * ((a.N + 15) / 16);
        if (strips <= (few ? 768 : 128) || (few && red >= 1024)) return MatmulKernel::kStream;
    }
    if (red >= 512 && tiles(a, 32) <= 256) return MatmulKernel::kSplit32;
    if (a.mode == kFwd && strips <= 768) return MatmulKernel::kStream;
    const int64_t tiles64 = tiles(a, 64);
    if (red >= 768 && tiles64 <= 256) return MatmulKernel::kTile64Parts;
    if (tiles64 <= 512) return MatmulKernel::kTile64;
    if (red >= 512 && tiles(a, 128) <= 256) return MatmulKernel::kTile128Deep;
    if (red < 512 || a.P < 128 * a.E) return MatmulKernel::kTile128;
    return MatmulKernel::kTile256;
}

}  // namespace moe
