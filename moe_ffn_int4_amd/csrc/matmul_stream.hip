// matmul_stream.hip -- y[s] = x[s] W_e^T for groups of a few rows, where reading the
// weights once is all that costs, and for small outputs, whose few blocks wait least here.
//
// A block takes strips of 16 weight rows (outputs n) and up to MX rows of x; its four waves
// split the reduction, each streaming its quarter through a ring of its own in LDS (no
// barrier, only the wave's own load counter), and their partial sums are added in
// order at the end. A chunk is KC values of the 16 weight rows and of the x rows,
// requested in 1 KB loads of whole rows' segments (KC * 2 bytes each: long
// contiguous pieces are what HBM wants) and multiplied by 16 x 16 x 32 products with
// the weight rows as D's rows. Rings are at most 80 KB a block, so that two blocks
// share a CU and one's start overlaps the other's stream.
//
// A launch has at most kMostBlocks blocks, each of which goes on to the next of its strips
// without a pause: its first chunks are requested before the strip in hand is summed. 16
// rows over E = 16 of 16384 x 5120, of which 8 experts have rows: 215 us, with a block a
// strip 249 (half of them find none); with 512, 1024 and 2048 blocks 220, 221 and 219. 64 rows
// over E = 16, 8192 x 4096: 171 (184; 176, 175, 174). Every expert with rows: 427 (430), 6.3 TB/s.
#include "matmul.h"

namespace moe {

namespace {

constexpr int kRowsN = 16;
constexpr int kWaves = 4;
constexpr int64_t kMostBlocks = 4096;

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
inline int ring_chunks(int64_t K) {
    const int64_t mine = (K + S::KC * kWaves - 1) / (S::KC * kWaves);
    return static_cast<int>(mine < S::RING ? mine : S::RING);
}

// A barrier for what is in LDS; requests stay in flight.
__device__ __forceinline__ void block_barrier_lds() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16-byte pieces of a segment XORed by this: a fragment read's 16 rows then touch
// 16 different groups of four banks (segments are multiples of 256 bytes)
__device__ __forceinline__ int seg_spread(int row) { return row & 15; }

}  // namespace

// The strips of a launch, 16 weight rows of one row tile each, are dealt to the blocks in
// turn. A wave's chunks of all its strips are one sequence, whose ring goes on from strip to strip.
template <typename S, Epilogue EPI>
__global__ __launch_bounds__(64 * kWaves, 2) void matmul_stream_kernel(MatmulArgs a, int rings) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr bool GATED = EPI == Epilogue::kGated;
    // one group of all rows: linear's, and a gated block's without offsets
    const bool dense = EPI == Epilogue::kLinear || (GATED && !a.offsets);
    RowTiles<S::MX> tiles;
    if (dense) tiles.total = static_cast<int>((a.P + S::MX - 1) / S::MX);
    else tiles.scan(a, lane);
    auto find = [&](int rt) __attribute__((always_inline)) {
        return dense ? dense_tile<S::MX>(a, rt) : tiles.find(rt, lane);
    };
    const int strips = static_cast<int>((a.N + kRowsN - 1) / kRowsN);
    const int stride = static_cast<int>(gridDim.x);
    // offsets out of order may give more strips than the host's bound: in rings that are
    // short of RING a block has one strip, and the numbers stay in 32 bits
    const int64_t all = static_cast<int64_t>(tiles.total) * strips, most = rings < S::RING ? stride : 1 << 30;
    const int total = static_cast<int>(all < most ? all : most);
    const int first = static_cast<int>(blockIdx.x);
    if (first >= total) return;

    const int K = static_cast<int>(a.K);
    // a wave's chunks of a strip: every kWaves-th
    const int chunks = (K + S::KC - 1) / S::KC;
    auto chunks_of = [&](int w) { return (chunks - w + kWaves - 1) / kWaves; };
    const int mine = chunks_of(wave);
    const uint8_t* ring = lds + wave * (S::kChunk * rings);
    const uint32_t ring_at = lds_address(ring);

    // a load covers kPerLoad rows: this lane's row in it, and its piece of the segment
    const int lrow = lane / S::kPieces, slot = lane % S::kPieces;
    // the strip whose chunks are being requested, and the next chunk of it
    const uint8_t *w, *x;
    uint32_t off[S::kLoads];
    int asked = first, ask = 0, ask_at = 0;
    auto open_strip = [&]() __attribute__((always_inline)) {
        const int rt = asked / strips, n0 = (asked - rt * strips) * (GATED ? kRowsN / 2 : kRowsN);
        const MatTile t = find(rt);
        const int nw = static_cast<int>(a.N - n0 < kRowsN ? a.N - n0 : kRowsN);
        w = reinterpret_cast<const uint8_t*>(
            uniform(reinterpret_cast<uint64_t>(a.b + (static_cast<int64_t>(t.group) * a.N + n0) * a.K)));
        x = reinterpret_cast<const uint8_t*>(uniform(reinterpret_cast<uint64_t>(a.a + t.row0 * a.K)));
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const bool isw = i < S::kLoadsW;
            const int r = (isw ? i : i - S::kLoadsW) * S::kPerLoad + lrow;
            const int most = isw ? nw : t.nrows;
            // a gated block's strip: eight gate rows and the up rows of the same outputs
            const int64_t row = GATED && isw ? (r & 7) + (r >> 3) * (a.N / 2) : r < most ? r : most - 1;
            off[i] = static_cast<uint32_t>(row * K * 2 + ((slot ^ seg_spread(r)) * 16));
        }
    };
    // the next chunk of this block's strips, if any
    auto request = [&]() __attribute__((always_inline)) {
        const int chunk = wave + ask * kWaves;
        const uint32_t to = ring_at + ask_at * S::kChunk;
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
        ask_at = ask_at == S::RING - 1 ? 0 : ask_at + 1;
        if (++ask == mine) {
            ask = 0;
            asked += stride;
            if (asked < total) open_strip();
        }
    };

    const int i16 = lane & 15, q = lane >> 4;
    const int xrow = i16 < S::MX ? i16 : S::MX - 1;
    int at = 0;    // ring place of the next chunk
    int done = 0;  // strips done
    if (mine > 0) open_strip();
#pragma unroll
    for (int c = 0; c < S::RING - 1; ++c)
        if (mine > 0 && asked < total) request();
    for (int strip = first; strip < total; strip += stride) {
        f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
        for (int c = 0; c < mine; ++c) {
            if (asked < total) {
                request();
                wait_loads<(S::RING - 1) * S::kLoads>();
            } else {
                wait_loads<0>();
            }
            const uint8_t* p = ring + at * S::kChunk;
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
            at = at == S::RING - 1 ? 0 : at + 1;
        }

        // the waves' sums, [row of x][n], each in the place of the wave's last chunk
        static_assert(16 * kRowsN * 4 <= S::kChunk, "sums fit a chunk");
        ++done;
        auto sums_of = [&](int v) {
            const int used = chunks_of(v) * done;
            return reinterpret_cast<float*>(lds + (v * rings + (used > 0 ? (used - 1) % S::RING : 0)) * S::kChunk);
        };
        *reinterpret_cast<f32x4*>(sums_of(wave) + i16 * kRowsN + 4 * q) = acc[0] + acc[1];
        block_barrier_lds();
        const int rt = strip / strips, n0 = (strip - rt * strips) * (GATED ? kRowsN / 2 : kRowsN);
        const MatTile t = find(rt);
        const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
        float v = sums_of(0)[m * kRowsN + n], up = 0.f;
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v += sums_of(i)[m * kRowsN + n];
        if constexpr (GATED) {
            up = sums_of(0)[m * kRowsN + (n | 8)];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) up += sums_of(i)[m * kRowsN + (n | 8)];
        }
        block_barrier_lds();
        if constexpr (GATED) {
            if (m < t.nrows && n < 8) store1_gated(a, t.row0 + m, n0 + n, v, up);
        } else {
            if (m < t.nrows && n0 + n < a.N) store1<EPI == Epilogue::kLinear>(a, t.row0 + m, a.N, n0 + n, v);
        }
    }
}

template <typename S, Epilogue EPI>
static hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
    static LdsDevices allowed;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(&matmul_stream_kernel<S, EPI>), S::kLds, allowed);
    if (e != hipSuccess) return e;
    const int64_t partial = a.E < a.P ? a.E : a.P;
    const int64_t strips = (a.P / S::MX + partial) * ((a.N + kRowsN - 1) / kRowsN);
    const int blocks = static_cast<int>(strips < kMostBlocks ? strips : kMostBlocks);
    const int rings = strips > kMostBlocks ? S::RING : ring_chunks<S>(a.K);
    hipLaunchKernelGGL((matmul_stream_kernel<S, EPI>), dim3(blocks), dim3(64 * kWaves),
                       S::kChunk * rings * kWaves, stream, a, rings);
    return hipGetLastError();
}

// The shape goes by the mean group, the sizes being unknown here. A group of more rows than MX
// streams its weights once for each MX of them: 512 rows over E = 128, 16384 x 5120, take 3.5 ms in
// groups of four, 2.9 with all rows in one group (tiles of 128 then: 0.11).
hipError_t launch_matmul_stream(Epilogue epilogue, const MatmulArgs& a, hipStream_t stream) {
    using Few = StreamShape<4, 256, 2>;
    using Many = StreamShape<16, 128, 2>;
    const bool few = a.P <= 4 * a.E;
    switch (epilogue) {
        case Epilogue::kLinear:
            return few ? launch<Few, Epilogue::kLinear>(a, stream) : launch<Many, Epilogue::kLinear>(a, stream);
        case Epilogue::kGated:
            return few ? launch<Few, Epilogue::kGated>(a, stream) : launch<Many, Epilogue::kGated>(a, stream);
        default: return few ? launch<Few, Epilogue::kPlain>(a, stream) : launch<Many, Epilogue::kPlain>(a, stream);
    }
}

}  // namespace moe
