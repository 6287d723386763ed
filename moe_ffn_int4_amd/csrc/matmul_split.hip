// matmul_split.hip -- the products of matmul.h for few outputs and long reductions, where a
// block's chain of steps is what takes the time.
//
// A block takes one tile of 32 x 32; its eight waves split the reduction, each taking every
// eighth 64-deep step of the whole tile through a ring of its own in LDS (no barrier, only the
// wave's own load counter), and their sums are added in order at the end. A CU then
// has 128 KB under way for half of the loads of a 64 x 64 tile. The wait for HBM, over a
// microsecond, bounds it: dx of 3 rows, 8704 x 136, takes 12 us (tiles of 64 in three parts 27,
// not split 52), dW of 7195 x 160 x 80 11 (25, 38).
#include "matmul.h"

namespace moe {

namespace {
constexpr int T = 32;
constexpr int kWaves = 8;
constexpr int kRing = 2;
constexpr int kTile = T * kStepR * 2;  // one operand of one step
constexpr int kStage = 2 * kTile;
constexpr int kLoads = kStage / 1024;  // a wave's, a step
constexpr int kLds = kWaves * kRing * kStage;
constexpr int kBand = 8;
}  // namespace

template <int MODE, Epilogue EPI>
__global__ __launch_bounds__(64 * kWaves, 2) void matmul_split_kernel(MatmulArgs a) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    MatTile t;
    int rt, ct;
    if (!find_tile<MODE, T, T, kBand>(a, lane, t, rt, ct)) return;
    const Operands<MODE> o = operands<MODE, T, T, EPI>(a, t, rt, ct, -1);

    constexpr bool AT = MODE == kDw, BT = MODE != kFwd;
    Stager<AT, T, 1> sa;
    Stager<BT, T, 1> sb;
    sa.init(o.a, o.lda, o.rows, 0, lane);
    sb.template init<EPI == Epilogue::kGated>(o.b, o.ldb, o.cols, 0, lane, a.N / 2);
    Reader<AT, T> ra;
    Reader<BT, T> rb;
    ra.init(0, lane);
    rb.init(0, lane);

    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int all = static_cast<int>((o.red + kStepR - 1) / kStepR);
    const int steps = (all - wave + kWaves - 1) / kWaves;  // this wave's
    const uint8_t* ring = lds + wave * (kRing * kStage);
    const uint32_t at = lds_address(ring);
    auto request = [&](int k) __attribute__((always_inline)) {
        const uint32_t to = at + (k % kRing) * kStage;
        sa.load(to, wave + k * kWaves, o.red);
        sb.load(to + kTile, wave + k * kWaves, o.red);
    };
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k)
        if (k < steps) request(k);
    for (int k = 0; k < steps; ++k) {
        if (k + kRing - 1 < steps) {
            request(k + kRing - 1);
            wait_loads<(kRing - 1) * kLoads>();
        } else {
            wait_loads<0>();
        }
        const uint8_t* p = ring + (k % kRing) * kStage;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) fa[i] = ra.read(p, i, s);
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[j] = rb.read(p + kTile, j, s);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mfma_bf16(fb[j], fa[i], acc[i][j]);
        }
        // the step is read before the request that overwrites it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }

    // the waves' sums, in order; each writes over its own ring, which it has read
    f32x4* sums = reinterpret_cast<f32x4*>(lds) + lane;
    constexpr int kEach = kRing * kStage / 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[wave * kEach + i * 64] = acc[i >> 1][i & 1];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] += sums[w * kEach + i * 64];
    store_all<MODE, EPI, 2, 1>(a, acc, Place{o.out_row, o.ldo, o.col0, o.rows, 0, o.cols},
                                  [&](int i) { return 16 * i; }, lane);
}

template <int MODE, Epilogue EPI>
static hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
    static LdsDevices allowed;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(&matmul_split_kernel<MODE, EPI>), kLds, allowed);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((matmul_split_kernel<MODE, EPI>), block_grid(matmul_blocks<MODE, T, T>(a)),
                       dim3(64 * kWaves), kLds, stream, a);
    return hipGetLastError();
}

hipError_t launch_matmul_split(int mode, Epilogue epilogue, const MatmulArgs& a, hipStream_t stream) {
    return with_mode(mode, epilogue,
                     [&](auto m, auto e) { return launch<decltype(m)::value, decltype(e)::value>(a, stream); });
}

}  // namespace moe
