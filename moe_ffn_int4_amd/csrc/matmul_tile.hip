// matmul_tile.hip -- the products of matmul.h in square tiles of 128 or 64, for outputs
// that do not fill the chip with 256 x 256 tiles, and the launch of the kernel that
// matmul_rule.h picks.
//
// One block of 4 waves in a 2 x 2 grid, each a quarter of the tile. The reduction runs
// in 64-deep steps through a ring of LDS stages: step k + RING - 1 is requested, straight
// to LDS, while step k is multiplied, one barrier a step. With 64 KB of LDS two blocks
// share a CU, and one block's loads and barriers overlap the other's products.
//
// KS parts of the reduction: a block of KS x 4 waves takes every KS-th step in each part,
// with a ring of its own, and adds the parts' sums in order. Few tiles leave a CU one
// block, whose steps then wait for HBM, at about 350 ns a step with three requested ahead: dx
// of 48 rows over 128 experts, 8896 x 232, about 160 tiles of 139 steps, takes 37 us with
// three parts and 53 without.
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

template <int MODE, Epilogue EPI, int T, int RING, int KS>
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
    const Operands<MODE> o = operands<MODE, T, T, EPI>(a, t, rt, ct, -1);

    constexpr bool AT = MODE == kDw, BT = MODE != kFwd;
    Stager<AT, T, kWaves> sa;
    Stager<BT, T, kWaves> sb;
    sa.init(o.a, o.lda, o.rows, wave, lane);
    sb.template init<EPI == Epilogue::kGated>(o.b, o.ldb, o.cols, wave, lane, a.N / 2);
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
    // holds of the others goes into rows that are not stored): dx of 30 rows, 16384 x 10240, 93.4 ->
    // 91.9 us, of 17, 2048 x 16384, 14.7 -> 14.5
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

    store_all<MODE, EPI, S, S / 2>(a, acc, Place{o.out_row, o.ldo, o.col0, o.rows, wn, o.cols},
                                      [&](int i) { return wm + 16 * i; }, lane);
}

template <int MODE, Epilogue EPI, int T, int RING, int KS>
static hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
    constexpr int kLds = KS * RING * 2 * T * kStepR * 2;
    static LdsDevices allowed;
    const hipError_t e = allow_lds(
        reinterpret_cast<const void*>(&matmul_tile_kernel<MODE, EPI, T, RING, KS>), kLds, allowed);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((matmul_tile_kernel<MODE, EPI, T, RING, KS>), block_grid(matmul_blocks<MODE, T, T>(a)),
                       dim3(64 * kWaves * KS), kLds, stream, a);
    return hipGetLastError();
}

template <int T, int RING, int KS>
static hipError_t launch_tile(int mode, Epilogue epilogue, const MatmulArgs& a, hipStream_t stream) {
    return with_mode(mode, epilogue, [&](auto m, auto e) {
        return launch<decltype(m)::value, decltype(e)::value, T, RING, KS>(a, stream);
    });
}

// The kernel that matmul_rule.h picks.
hipError_t launch_matmul(int mode, Epilogue epilogue, const MatmulArgs& a, hipStream_t stream) {
    switch (choose_matmul(MatmulSizes{mode, a.P, a.E, a.N, a.K})) {
        case MatmulKernel::kStream: return launch_matmul_stream(epilogue, a, stream);
        case MatmulKernel::kSplit32: return launch_matmul_split(mode, epilogue, a, stream);
        case MatmulKernel::kTile64Parts: return launch_tile<64, 3, 3>(mode, epilogue, a, stream);
        case MatmulKernel::kTile64: return launch_tile<64, 4, 1>(mode, epilogue, a, stream);
        case MatmulKernel::kTile128Deep: return launch_tile<128, 4, 1>(mode, epilogue, a, stream);
        case MatmulKernel::kTile128: return launch_tile<128, 2, 1>(mode, epilogue, a, stream);
        case MatmulKernel::kTile256: return launch_matmul256(mode, epilogue, a, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace moe
