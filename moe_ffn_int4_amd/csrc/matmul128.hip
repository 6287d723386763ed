// matmul128.hip -- the products of matmul.h in 128 x 128 tiles.
//
// One block of 4 waves in a 2 x 2 grid, each 64 x 64 of the output (4 x 4 products
// of 16 x 16 x 32, 64 accumulators a lane). The reduction runs in 64-deep steps
// through two 32 KB LDS stages: the loads of step k + 1 go straight to LDS while
// step k is multiplied, one barrier a step. 64 KB of LDS lets two blocks share a
// CU, and one block's loads and barriers overlap the other's products.
#include "matmul.h"

namespace moe {

namespace {
constexpr int BM = 128;
constexpr int BN = 128;
constexpr int kWaves = 4;
constexpr int kTile = BM * kStepR * 2;      // 16 KB: one operand of one step
constexpr int kStage = 2 * kTile;
constexpr int kBand = 8;                    // row tiles walked down a column of tiles
}  // namespace

template <int MODE, bool LINEAR>
__global__ __launch_bounds__(64 * kWaves, 2) void matmul128_kernel(MatmulArgs a) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ncol = static_cast<int>(((MODE == kFwd ? a.N : a.K) + BN - 1) / BN);

    MatTile t;
    int rt, ct;
    if (MODE == kDw) {
        // every group has the same tiles; each XCD takes a contiguous eighth of them
        const int nrow = static_cast<int>((a.N + BM - 1) / BM);
        const int64_t n = static_cast<int64_t>(nrow) * ncol, slots = (n + 7) / 8;
        t.group = static_cast<int>(blockIdx.x / (8 * slots));
        const int64_t local = blockIdx.x - t.group * 8 * slots;
        const int64_t lin = (local & 7) * slots + (local >> 3);
        if (lin >= n) return;
        band_walk<kBand>(lin, nrow, ncol, rt, ct);
        group_rows(a, t.group, t.row0, t.nrows);
        if (a.accumulate && t.nrows == 0) return;
    } else {
        RowTiles<BM> tiles;
        tiles.scan(a, lane);
        int64_t lin;
        if (!xcd_slot(static_cast<int64_t>(tiles.total) * ncol, lin)) return;
        band_walk<kBand>(lin, tiles.total, ncol, rt, ct);
        t = tiles.find(rt, lane);
    }
    const Operands<MODE> o = operands<MODE, BM, BN>(a, t, rt, ct);

    constexpr bool AT = MODE == kDw, BT = MODE != kFwd;
    Stager<AT, false, BM, kWaves> sa;
    Stager<BT, true, BN, kWaves> sb;
    sa.init(o.a, o.lda, o.rows, wave, lane);
    sb.init(o.b, o.ldb, o.cols, wave, lane);
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    Reader<AT, false, BM> ra;
    Reader<BT, true, BN> rb;
    ra.init(wm, lane);
    rb.init(wn, lane);

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int steps = static_cast<int>((o.red + kStepR - 1) / kStepR);
    const uint32_t at = lds_address(lds);
    if (steps > 0) {
        sa.load(at, 0, o.red);
        sb.load(at + kTile, 0, o.red);
    }
    for (int k = 0; k < steps; ++k) {
        const uint8_t* cur = lds + (k & 1) * kStage;
        const uint32_t next = at + (~k & 1) * kStage;
        // step k has landed and every wave has read step k - 1
        wait_loads<0>();
        __syncthreads();
        if (k + 1 < steps) {
            sa.load(next, k + 1, o.red);
            sb.load(next + kTile, k + 1, o.red);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            bf16x8 fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i] = ra.read(cur, i, s);
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[j] = rb.read(cur + kTile, j, s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = mfma_bf16(fb[j], fa[i], acc[i][j]);
        }
    }

    const int i16 = lane & 15, q = lane >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = wm + 16 * i + i16;
        if (row >= o.rows) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int col = wn + 16 * q + 8 * h;
            if (col >= o.cols) continue;
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = acc[i][2 * h + (r >> 2)][r & 3];
            store8<LINEAR>(a, o.out_row + row, o.ldo, o.col0 + col, v);
        }
    }
}

template <int MODE, bool LINEAR>
static hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
    const int64_t ncol = ((MODE == kFwd ? a.N : a.K) + BN - 1) / BN;
    int64_t blocks;
    if (MODE == kDw) {
        blocks = a.E * 8 * ((((a.N + BM - 1) / BM) * ncol + 7) / 8);
    } else {
        // row tiles: full ones and at most one partial tile for each group with rows
        const int64_t partial = a.E < a.P ? a.E : a.P;
        blocks = 8 * ((a.P / BM + partial) * ncol / 8 + 1);
    }
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((matmul128_kernel<MODE, LINEAR>), dim3(static_cast<unsigned>(blocks)),
                       dim3(64 * kWaves), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_matmul128(int mode, bool linear, const MatmulArgs& a, hipStream_t stream) {
    if (mode == kDx) return launch<kDx, false>(a, stream);
    if (mode == kDw) return launch<kDw, false>(a, stream);
    return linear ? launch<kFwd, true>(a, stream) : launch<kFwd, false>(a, stream);
}

hipError_t launch_matmul(int mode, bool linear, const MatmulArgs& a, hipStream_t stream) {
    return launch_matmul128(mode, linear, a, stream);
}

}  // namespace moe
