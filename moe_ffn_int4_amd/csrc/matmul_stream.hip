// matmul_stream.hip -- y[s] = x[s] W_e^T for groups of a few rows, where reading the
// weights once is all that costs, and for small outputs, whose few blocks wait least here.
//
// A block takes 16 weight rows (outputs n) and up to MX rows of x; its four waves
// split the reduction, each streaming its quarter through a ring of its own in LDS (no
// barrier, only the wave's own load counter), and their partial sums are added in
// order at the end. A chunk is KC values of the 16 weight rows and of the x rows,
// requested in 1 KB loads of whole rows' segments (KC * 2 bytes each: long
// contiguous pieces are what HBM wants) and multiplied by 16 x 16 x 32 products with
// the weight rows as D's rows. Rings are at most 80 KB a block, so that two blocks
// share a CU and one's start overlaps the other's stream.
#include "matmul.h"

namespace moe {

namespace {

constexpr int kRowsN = 16;
constexpr int kWaves = 4;

// MX: most rows of x; KC: values of a chunk; RING: chunks in LDS
template <int MX_, int KC_, int RING_>
struct StreamShape {
    static constexpr int MX = MX_, KC = KC_, RING = RING_;
    static constexpr int kSeg = KC * 2;                     // bytes of a row's segment
    static constexpr int kPerLoad = 1024 / kSeg;            // rows a 1 KB load
    static constexpr int kLoadsW = kRowsN / kPerLoad;
    static constexpr int kLoadsX = (MX + kPerLoad - 1) / kPerLoad;
    static constexpr int kLoads = kLoadsW + kLoadsX;
    static constexpr int kChunk = kLoads * 1024;
    static constexpr int kLds = kChunk * RING * kWaves;
    static constexpr int kPieces = kSeg / 16;
};

// Chunks a wave's ring holds: a short reduction has fewer, and its blocks more room on
// a CU.
template <typename S>
__host__ __device__ inline int ring_chunks(int64_t K) {
    const int64_t mine = (K + S::KC * kWaves - 1) / (S::KC * kWaves);
    return static_cast<int>(mine < S::RING ? mine : S::RING);
}

// 16-byte pieces of a segment XORed by this: a fragment read's 16 rows then touch
// 16 different groups of four banks (segments are multiples of 256 bytes)
__device__ __forceinline__ int seg_spread(int row) { return row & 15; }

}  // namespace

template <typename S, bool LINEAR>
__global__ __launch_bounds__(64 * kWaves, 2) void matmul_stream_kernel(MatmulArgs a) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    RowTiles<S::MX> tiles;
    tiles.scan(a, lane);
    // blocks: the row tiles' 16-row strips of weights, tile after tile
    const int strips = static_cast<int>((a.N + kRowsN - 1) / kRowsN);
    const int block = static_cast<int>(block_index()), rt = block / strips;
    if (rt >= tiles.total) return;
    const int n0 = (block - rt * strips) * kRowsN;
    const MatTile t = tiles.find(rt, lane);
    const int nw = static_cast<int>(a.N - n0 < kRowsN ? a.N - n0 : kRowsN);

    const uint8_t* w = reinterpret_cast<const uint8_t*>(
        a.b + (static_cast<int64_t>(t.group) * a.N + n0) * a.K);
    const uint8_t* x = reinterpret_cast<const uint8_t*>(a.a + t.row0 * a.K);
    const int K = static_cast<int>(a.K);
    // this wave's chunks: every kWaves-th
    const int chunks = (K + S::KC - 1) / S::KC;
    const int mine = (chunks - wave + kWaves - 1) / kWaves;
    const int rings = ring_chunks<S>(K);
    const uint8_t* ring = lds + wave * (S::kChunk * rings);
    const uint32_t ring_at = lds_address(ring);

    // a load covers kPerLoad rows: this lane's row in it, and its piece of the segment
    const int lrow = lane / S::kPieces, slot = lane % S::kPieces;
    uint32_t off[S::kLoads];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
        const bool isw = i < S::kLoadsW;
        const int r = (isw ? i : i - S::kLoadsW) * S::kPerLoad + lrow;
        const int most = isw ? nw : t.nrows;
        off[i] = static_cast<uint32_t>((r < most ? r : most - 1) * K * 2 + ((slot ^ seg_spread(r)) * 16));
    }
    auto request = [&](int c) __attribute__((always_inline)) {
        const int chunk = wave + c * kWaves;
        const uint32_t to = ring_at + (c % S::RING) * S::kChunk;
        const int left = K - chunk * S::KC;
        const uint8_t* wc = w + static_cast<int64_t>(chunk) * S::kSeg;
        const uint8_t* xc = x + static_cast<int64_t>(chunk) * S::kSeg;
        if (left >= S::KC) {
#pragma unroll
            for (int i = 0; i < S::kLoads; ++i)
                lds_load16(i < S::kLoadsW ? wc : xc, off[i], to + i * 1024);
        } else {
#pragma unroll
            for (int i = 0; i < S::kLoads; ++i) {
                const int r = (i < S::kLoadsW ? i : i - S::kLoadsW) * S::kPerLoad + lrow;
                const int at = (slot ^ seg_spread(r)) * 8;
                const void* src = at < left ? static_cast<const void*>((i < S::kLoadsW ? wc : xc) + off[i])
                                            : static_cast<const void*>(g_zero16);
                lds_load16(src, to + i * 1024);
            }
        }
    };

    const int i16 = lane & 15, q = lane >> 4;
    const int xrow = i16 < S::MX ? i16 : S::MX - 1;
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int c = 0; c < S::RING - 1; ++c)
        if (c < mine) request(c);
    for (int c = 0; c < mine; ++c) {
        if (c + S::RING - 1 < mine) {
            request(c + S::RING - 1);
            wait_loads<(S::RING - 1) * S::kLoads>();
        } else {
            wait_loads<0>();
        }
        const uint8_t* p = ring + (c % S::RING) * S::kChunk;
#pragma unroll
        for (int s = 0; s < S::KC / 32; ++s) {
            const bf16x8 fw = *reinterpret_cast<const bf16x8*>(
                p + i16 * S::kSeg + (((4 * s + q) ^ seg_spread(i16)) * 16));
            const bf16x8 fx = *reinterpret_cast<const bf16x8*>(
                p + S::kLoadsW * 1024 + xrow * S::kSeg + (((4 * s + q) ^ seg_spread(xrow)) * 16));
            acc[s & 1] = mfma_bf16(fw, fx, acc[s & 1]);
        }
        // the chunk is read before the request that overwrites it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }

    // waves' sums: [wave][row of x][n]
    __syncthreads();
    static_assert(kWaves * 16 * kRowsN * 4 <= S::kChunk * kWaves, "sums fit the rings");
    float* part = reinterpret_cast<float*>(lds);
    *reinterpret_cast<f32x4*>(part + (wave * 16 + i16) * kRowsN + 4 * q) = acc[0] + acc[1];
    __syncthreads();
    const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
    if (m >= t.nrows || n >= nw) return;
    float v = part[m * kRowsN + n];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) v += part[(i * 16 + m) * kRowsN + n];
    store1<LINEAR>(a, t.row0 + m, a.N, n0 + n, v);
}

template <typename S, bool LINEAR>
static hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
    static const hipError_t ready = hipFuncSetAttribute(
        reinterpret_cast<const void*>(&matmul_stream_kernel<S, LINEAR>),
        hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (ready != hipSuccess) return ready;
    const int64_t partial = a.E < a.P ? a.E : a.P;
    const int64_t blocks = (a.P / S::MX + partial) * ((a.N + kRowsN - 1) / kRowsN);
    hipLaunchKernelGGL((matmul_stream_kernel<S, LINEAR>), block_grid(blocks), dim3(64 * kWaves),
                       S::kChunk * ring_chunks<S>(a.K) * kWaves, stream, a);
    return hipGetLastError();
}

hipError_t launch_matmul_stream(bool linear, const MatmulArgs& a, hipStream_t stream) {
    using Few = StreamShape<4, 256, 2>;
    using Many = StreamShape<16, 128, 2>;
    if (a.P <= 4 * a.E) return linear ? launch<Few, true>(a, stream) : launch<Few, false>(a, stream);
    return linear ? launch<Many, true>(a, stream) : launch<Many, false>(a, stream);
}

}  // namespace moe
