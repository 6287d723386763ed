// matmul_tile.hip -- the products of matmul.h in square tiles of 128 or 64, for outputs
// that do not fill the chip with 256 x 256 tiles, and the choice among all the kernels.
//
// One block of 4 waves in a 2 x 2 grid, each a quarter of the tile. The reduction runs
// in 64-deep steps through a ring of LDS stages: step k + RING - 1 is requested, straight
// to LDS, while step k is multiplied, one barrier a step. With 64 KB of LDS two blocks
// share a CU, and one block's loads and barriers overlap the other's products.
//
// KS parts of the reduction: a block of KS x 4 waves takes every KS-th step in each part,
// with a ring of its own, and adds the parts' sums in order. Few tiles leave a CU one
// block, whose steps then wait for HBM: 17 x 64 x 5120, a single tile, takes 350 ns a
// step with three requested ahead, and 20 us instead of 28 with three parts.
#include "matmul.h"

namespace moe {

namespace {
constexpr int kWaves = 4;
constexpr int kBand = 8;  // row tiles walked down a column of tiles

// at most `steps` of the youngest steps' requests (PER a wave each) left in flight
template <int PER, int MOST>
__device__ __forceinline__ void wait_steps(int steps) {
    if constexpr (MOST == 0) {
        wait_loads<0>();
    } else {
        if (steps >= MOST) wait_loads<PER * MOST>();
        else wait_steps<PER, MOST - 1>(steps);
    }
}
}  // namespace

template <int MODE, bool LINEAR, int T, int RING, int KS>
__global__ __launch_bounds__(64 * kWaves * KS, KS == 1 ? 2 : KS) void matmul_tile_kernel(MatmulArgs a) {
    constexpr int kTile = T * kStepR * 2;  // one operand of one step
    constexpr int kStage = 2 * kTile;
    constexpr int S = T / 32;              // 16-wide sub-tiles of a wave, each way
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & (kWaves - 1);
    const int part = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * kWaves));
    MatTile t;
    int rt, ct;
    if (!find_tile<MODE, T, T, kBand>(a, lane, t, rt, ct)) return;
    const Operands<MODE> o = operands<MODE, T, T>(a, t, rt, ct, -1);

    constexpr bool AT = MODE == kDw, BT = MODE != kFwd;
    Stager<AT, T, kWaves> sa;
    Stager<BT, T, kWaves> sb;
    sa.init(o.a, o.lda, o.rows, wave, lane);
    sb.init(o.b, o.ldb, o.cols, wave, lane);
    const int wm = (wave >> 1) * (T / 2), wn = (wave & 1) * (T / 2);
    Reader<AT, T> ra;
    Reader<BT, T> rb;
    ra.init(wm, lane);
    rb.init(wn, lane);

    f32x4 acc[S][S];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < S; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int all = static_cast<int>((o.red + kStepR - 1) / kStepR);
    const int steps = (all - part + KS - 1) / KS, most = (all + KS - 1) / KS;  // this part's, and any's
    const uint8_t* ring = lds + part * (RING * kStage);
    const uint32_t at = lds_address(ring);
    constexpr int kLoads = 2 * T / 8 / kWaves;  // a wave's, a step
    // A's first 32 rows alone where the tile has no more (a wave's first load of two; what LDS
    // holds of the others goes into rows that are not stored): 17 x 16384 x 5120 dx 53.7 -> 51.4 us
    const bool half = MODE != kDw && T == 64 && o.rows <= 32;
    auto request = [&](int stage, int k) __attribute__((always_inline)) {
        if (half) sa.template load<0, T / 64>(at + stage * kStage, part + k * KS, o.red);
        else sa.load(at + stage * kStage, part + k * KS, o.red);
        sb.load(at + stage * kStage + kTile, part + k * KS, o.red);
    };
    for (int k = 0; k < RING - 1 && k < steps; ++k) request(k, k);
    int cur = 0, next = RING - 1;  // stages of step k and of step k + RING - 1
    for (int k = 0; k < most; ++k) {
        // step k has landed (steps k + 1 .. k + RING - 2 may be under way), and every
        // wave has read step k - 1, whose stage is the next to be written
        if (half) wait_steps<kLoads - T / 64, RING - 2>(steps - 1 - k);
        else wait_steps<kLoads, RING - 2>(steps - 1 - k);
        __syncthreads();
        if (KS > 1 && k >= steps) break;  // the last round, of fewer parts
        if (k + RING - 1 < steps) request(next, k + RING - 1);
        const uint8_t* p = ring + cur * kStage;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 fa[S], fb[S];
#pragma unroll
            for (int i = 0; i < S; ++i) fa[i] = ra.read(p, i, s);
#pragma unroll
            for (int j = 0; j < S; ++j) fb[j] = rb.read(p + kTile, j, s);
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int j = 0; j < S; ++j) acc[i][j] = mfma_bf16(fb[j], fa[i], acc[i][j]);
        }
        cur = cur == RING - 1 ? 0 : cur + 1;
        next = next == RING - 1 ? 0 : next + 1;
    }

    if (KS > 1) {
        // the other parts' sums, in order, through LDS
        __syncthreads();
        f32x4* sums = reinterpret_cast<f32x4*>(lds) + threadIdx.x % (64 * kWaves);
#pragma unroll
        for (int p = 1; p < KS; ++p) {
            f32x4* mine = sums + (p - 1) * (S * S * 64 * kWaves);
            if (part == p) {
#pragma unroll
                for (int i = 0; i < S * S; ++i) mine[i * 64 * kWaves] = acc[i / S][i % S];
            }
        }
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int p = 1; p < KS; ++p)
#pragma unroll
            for (int i = 0; i < S * S; ++i) acc[i / S][i % S] += sums[((p - 1) * S * S + i) * 64 * kWaves];
    }

    store_all<MODE, LINEAR, S, S / 2>(a, acc, Place{o.out_row, o.ldo, o.col0, o.rows, wn, o.cols},
                                      [&](int i) { return wm + 16 * i; }, lane);
}

template <int MODE, bool LINEAR, int T, int RING, int KS>
static hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
    constexpr int kLds = KS * RING * 2 * T * kStepR * 2;
    static const hipError_t ready = hipFuncSetAttribute(
        reinterpret_cast<const void*>(&matmul_tile_kernel<MODE, LINEAR, T, RING, KS>),
        hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (ready != hipSuccess) return ready;
    const int64_t blocks = matmul_blocks<MODE, T, T>(a);
    if (blocks > 2 * kGridX) return hipErrorInvalidConfiguration;  // 256 threads each
    hipLaunchKernelGGL((matmul_tile_kernel<MODE, LINEAR, T, RING, KS>), dim3(static_cast<unsigned>(blocks)),
                       dim3(64 * kWaves * KS), kLds, stream, a);
    return hipGetLastError();
}

template <int T, int RING, int KS>
static hipError_t launch_tile(int mode, bool linear, const MatmulArgs& a, hipStream_t stream) {
    if (mode == kDx) return launch<kDx, false, T, RING, KS>(a, stream);
    if (mode == kDw) return launch<kDw, false, T, RING, KS>(a, stream);
    return linear ? launch<kFwd, true, T, RING, KS>(a, stream) : launch<kFwd, false, T, RING, KS>(a, stream);
}

// Row tiles of T, an estimate where the host does not know the group sizes: each group's
// last one is half empty.
static int64_t row_tiles(const MatmulArgs& a, int64_t T) {
    const int64_t groups = a.E < a.P ? a.E : a.P;
    return groups == 1 ? (a.P + T - 1) / T : a.P / T + (groups + 1) / 2;
}

static int64_t tiles(int mode, const MatmulArgs& a, int64_t T) {
    auto up = [T](int64_t v) { return (v + T - 1) / T; };
    if (mode == kDw) return a.E * up(a.N) * up(a.K);
    return row_tiles(a, T) * up(mode == kFwd ? a.N : a.K);
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
//     19.2); dx of 48 rows over E = 128, 8896 x 232 (about 500): 54.6 (38.7).
//   * y = x W^T of up to 768 streaming blocks: those. 496 x 120 x 5328 (248): 10.0 against
//     21.7 in tiles of 64, split.
//   * up to 256 tiles of 64 and a reduction of 768 or more: those, split in three. 100 x
//     4096 x 4096 (128 tiles): 16.1 against 23.5 not split, 18.4 split in two; 256 x 4096 x
//     4096 (256): 21.6 (24.5); 17 x 16384 x 5120, dx (80): 51 (79); 256 x 8192 x 5120 (512):
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
// Over 2700 products of random sizes this takes 2 % longer than the best kernel for each.
hipError_t launch_matmul(int mode, bool linear, const MatmulArgs& a, hipStream_t stream) {
    const int64_t red = mode == kFwd ? a.K : mode == kDx ? a.N : a.P / a.E;
    const bool few = a.P <= 16 || a.P <= 4 * a.E;
    int64_t strips = 0;  // blocks of the streaming kernel
    if (mode == kFwd) {
        strips = row_tiles(a, a.P <= 4 * a.E ? 4 : 16) * ((a.N + 15) / 16);
        if (strips <= (few ? 768 : 128) || (few && red >= 1024)) return launch_matmul_stream(linear, a, stream);
    }
    if (red >= 512 && tiles(mode, a, 32) <= 256) return launch_matmul_split(mode, linear, a, stream);
    if (mode == kFwd && strips <= 768) return launch_matmul_stream(linear, a, stream);
    const int64_t tiles64 = tiles(mode, a, 64);
    if (red >= 768 && tiles64 <= 256) return launch_tile<64, 3, 3>(mode, linear, a, stream);
    if (tiles64 <= 512) return launch_tile<64, 4, 1>(mode, linear, a, stream);
    if (red >= 512 && tiles(mode, a, 128) <= 256) return launch_tile<128, 4, 1>(mode, linear, a, stream);
    if (red < 512 || a.P < 128 * a.E) return launch_tile<128, 2, 1>(mode, linear, a, stream);
    return launch_matmul256(mode, linear, a, stream);
}

}  // namespace moe
