// int4.hip -- products with 4-bit weights, y[s] = x[s] (scale * code)^T, from a single row to
// tiles of 64 rows.
//
// The reduction runs in steps of 128, one tile column of the weights' tiled order: a strip of 16
// features is 1 KB of codes and 64 S bytes of scales a step (S = 128 / group), both contiguous, and
// goes straight from HBM to LDS, as do 256 bytes of each row of x. A ring of stages keeps the next
// steps under way. KS parts of the reduction, each a group of waves with a ring of its own,
// take every KS-th step and add their sums in order at the end: a product of few rows has few
// blocks, and more of its weights are then on their way at once.
//
// Codes reach the matrix cores exactly, as the bf16 numbers 16 + u, u = code + 8, which are the bits of
// 16 with the nibble at the top of the mantissa. A group's sum of x * (16 + u) starts from -24 sum x, which
// one more matrix instruction against the constant -24 gives for each fragment of x, shared by all
// strips of a wave; what is left is the sum of x * code, in fp32, which the group's fp32 scale multiplies into
// the accumulator. So no weight is ever rounded. (128 + u, the nibble at the bottom, saves a shift for eight
// codes, but the sums that cancel are then over 136 |x|.) What cancels is 24 sum |x|, so that errors go by sum |x scale| and not by
// sum |x scale code|: 2^-17 of it at most, as measured.
//
// A wave multiplies MT sub-tiles of 16 rows by NS strips. Weights come first in the instruction, so that a lane holds four
// consecutive columns of one row, as in matmul.h, whose stores the larger tiles use.
//
// Steps of 128 are what one column of the tiled order has, so that every load is of a whole kilobyte. One row of
// 8192 x 5120 takes 8 us (launch and one wait for HBM), 16 rows over 16 groups, 16384 x 5120, 79 to 93 us (5 to 5.8 TB/s, bound
// by the requests to LDS). Tens of rows are bound by the eight instructions of a widening, which a tile of 16 rows repeats for each 16
// (37 x 5120 x 8192 13.7 us); thousands by matrix instructions, a fifth of them the correction's, as these and other vector
// instructions hardly overlap on a SIMD (4096 x 5120 x 8192 312 us, 1100 TFLOP/s; groups of 64 350, of 32 406;
// 342 on the slowest of four boxes).
#include "int4.h"

#include "matmul.h"

namespace moe {

namespace {

constexpr int kDepth = 128;  // of a step
constexpr int kBand = 8;

// ROWS of x in a tile; each of KS parts has WAVES waves, which take NS strips each; RING stages
template <int ROWS_, int WAVES_, int NS_, int KS_, int RING_>
struct Shape {
    static constexpr int ROWS = ROWS_, WAVES = WAVES_, NS = NS_, KS = KS_, RING = RING_;
    static constexpr int MT = (ROWS + 15) / 16;                     // sub-tiles of rows, all of them every wave's
    static constexpr int kStrips = WAVES * NS, COLS = 16 * kStrips;
    static constexpr int kThreads = 64 * WAVES * KS;
    static constexpr int kRowsMine = ROWS / WAVES;                  // rows of x that a wave requests, beside its strips
    static constexpr int kLoadsX = kRowsMine > 4 ? kRowsMine / 4 : 1;
    static constexpr int kLoads = kLoadsX + NS + 1;                 // a wave's, a step
    // sums meet in LDS before they are stored: of several parts, and of a single sub-tile, whose rows are not whole stores
    static constexpr bool kJoin = KS > 1 || MT == 1;
    static constexpr int kX = ROWS * kDepth * 2, kW = kStrips * 1024;
    static constexpr int stage(int S) { return kX + kW + kStrips * 64 * S; }
    static constexpr int kSumRow = COLS * 4 + 16;                   // bytes, of the parts' sums
    static constexpr int lds(int S) {
        const int ring = KS * RING * stage(S), sums = kJoin ? KS * 16 * MT * kSumRow : 0;
        return ring > sums ? ring : sums;
    }
    // waves of a SIMD, as LDS allows: the compiler need not save registers for more (without this it reads a step's codes one
    // by one, 100 x 5120 x 8192 24.0 us against 22.1); at least two, so that sums stay in ordinary registers
    static constexpr int simd_waves(int S) { return 160 * 1024 / lds(S) * kThreads / 256; }
    static_assert(kRowsMine * WAVES == ROWS && (kRowsMine <= 4 || kRowsMine % 4 == 0), "rows are dealt evenly");
    static_assert(lds(4) <= 160 * 1024, "LDS");
};

// The order of a row's 16-byte pieces of x in LDS is XORed by this, so that the 16 lanes that are served
// together, of 16 rows (half of them of the next quarter), touch different banks.
template <int S>
__device__ __forceinline__ int spread(int row) {
    return S == 1 ? (row & 3) << 2 | (row >> 2 & 3) : row & 15;
}

// 8 codes -> bf16 pairs 16 + u in order. A byte times 2^3 + 2^15 has its nibbles at bits 3 and 19 (one instruction, which
// picks the byte); a nibble's top bit flipped is u's, and it and the bits of 16 are one XOR (one more, with the mask).
__device__ __forceinline__ bf16x8 offset_codes(uint32_t w) {
    constexpr uint32_t kMask = 0x00780078u, kFlip = 0x41C041C0u;  // bf16 16.0 | 0x40, twice
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = (__umul24(w >> 8 * j & 0xFF, 0x8008) & kMask) ^ kFlip;
    return __builtin_bit_cast(bf16x8, r);
}

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

template <typename Sh, bool LINEAR, int S>
__global__ __launch_bounds__(Sh::kThreads)
__attribute__((amdgpu_waves_per_eu(2, Sh::simd_waves(S)))) void int4_kernel(Int4Args args) {
    constexpr int ROWS = Sh::ROWS, MT = Sh::MT, NS = Sh::NS, KS = Sh::KS, RING = Sh::RING;
    constexpr int kStage = Sh::stage(S);
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const MatmulArgs& a = args.m;
    const int lane = threadIdx.x & 63;
    const int all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = all_waves % Sh::WAVES, part = all_waves / Sh::WAVES;
    MatTile t;
    int rt, ct;
    if (!find_tile<kFwd, ROWS, Sh::COLS, kBand>(a, lane, t, rt, ct)) return;

    const int tiles = static_cast<int>(a.K) / kDepth;  // of a strip
    const int strips = static_cast<int>(a.N / 16) - ct * Sh::kStrips;  // valid, from the tile's first
    const int64_t strip0 = static_cast<int64_t>(t.group) * (a.N / 16) + static_cast<int64_t>(ct) * Sh::kStrips;
    const uint8_t* q = reinterpret_cast<const uint8_t*>(
        uniform(reinterpret_cast<uint64_t>(args.q + strip0 * tiles * 1024)));
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(
        uniform(reinterpret_cast<uint64_t>(args.scales + strip0 * tiles * 16 * S)));
    const uint8_t* x = reinterpret_cast<const uint8_t*>(uniform(reinterpret_cast<uint64_t>(a.a + t.row0 * a.K)));

    // this lane's sources at step 0, past the end the last valid ones: what they give is dropped
    uint32_t off_x[Sh::kLoadsX];
#pragma unroll
    for (int i = 0; i < Sh::kLoadsX; ++i) {
        const int r = wave * Sh::kRowsMine + 4 * i + (lane >> 4);
        const int from = r < t.nrows ? r : t.nrows - 1;
        off_x[i] = static_cast<uint32_t>(from * static_cast<int>(a.K) * 2 + (((lane & 15) ^ spread<S>(r)) * 16));
    }
    int64_t strip_q[NS];  // uniform
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int s = wave * NS + i;
        strip_q[i] = static_cast<int64_t>(s < strips ? s : strips - 1) * tiles * 1024;
    }
    const int s_strip = wave * NS + lane / (4 * S);
    const uint8_t* my_sc = sc + static_cast<int64_t>(s_strip < strips ? s_strip : strips - 1) * tiles * 64 * S +
                           (lane % (4 * S)) * 16;
    const int steps = (tiles - part + KS - 1) / KS, most = (tiles + KS - 1) / KS;  // this part's, and any's
    const int turn = ct % tiles;
    const uint8_t* ring = lds + part * (RING * kStage);
    const uint32_t ring_at = lds_address(ring);
    auto request = [&](int stage, int k) __attribute__((always_inline)) {
        int g = part + k * KS;
        if (KS == 1) g = g + turn < tiles ? g + turn : g + turn - tiles;
        const uint32_t at = ring_at + stage * kStage;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            lds_load16(q + strip_q[i] + static_cast<int64_t>(g) * 1024, lane * 16,
                       at + Sh::kX + (wave * NS + i) * 1024);
        if (lane < NS * 4 * S)
            lds_load16(my_sc + static_cast<int64_t>(g) * 64 * S,
                       at + Sh::kX + Sh::kW + wave * NS * 64 * S);
        if (Sh::kRowsMine >= 4 || lane < 16 * Sh::kRowsMine) {
#pragma unroll
            for (int i = 0; i < Sh::kLoadsX; ++i)
                lds_load16(x + g * (kDepth * 2), off_x[i], at + (wave * Sh::kRowsMine + 4 * i) * (kDepth * 2));
        }
    };
    for (int k = 0; k < RING - 1 && k < steps; ++k) request(k, k);

    const int i16 = lane & 15, qd = lane >> 4;
    const int xrow = i16 < ROWS ? i16 : ROWS - 1;
    const u32x4 minus = {0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};  // bf16 -24
    f32x4 acc[MT][NS];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NS; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    int cur = 0, next = RING - 1;  // stages of step k and of step k + RING - 1
    for (int k = 0; k < most; ++k) {
        // step k has landed, and every wave has read step k - 1, whose stage is the next to be written
        wait_steps<Sh::kLoads, RING - 2>(steps - 1 - k);
        __syncthreads();
        if (KS > 1 && k >= steps) break;  // the last round, of fewer parts
        if (k + RING - 1 < steps) request(next, k + RING - 1);
        const uint8_t* p = ring + cur * kStage;
        const uint8_t* px = p + xrow * (kDepth * 2);
        // Which of a group's columns a lane's fragment has is free, as long as x and codes agree: with groups of 128 a lane
        // takes its quarter's 32 codes in one read, with smaller ones eight of each slice
        const uint8_t* pw = p + Sh::kX + wave * NS * 1024 + i16 * 16 + qd * (S == 1 ? 256 : 4);
        const float* ps = reinterpret_cast<const float*>(p + Sh::kX + Sh::kW + wave * NS * 64 * S) + 4 * qd * S;
        constexpr int PER = 4 / S;  // 32-deep slices of a group
        // the scales of this lane's four features stand together, S each; where registers allow, all of them are
        // read at once, 16 bytes at a time
        constexpr bool AHEAD = NS * S <= (MT <= 2 ? 16 : 8);
        f32x4 all[AHEAD ? NS * S : 1];
        if constexpr (AHEAD) {
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int v = 0; v < S; ++v) all[j * S + v] = *reinterpret_cast<const f32x4*>(ps + j * 16 * S + 4 * v);
        }
#pragma unroll
        for (int g = 0; g < S; ++g) {
            bf16x8 fx[PER][MT];
#pragma unroll
            for (int s = 0; s < PER; ++s)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    fx[s][i] = *reinterpret_cast<const bf16x8*>(px + i * 16 * (kDepth * 2) +
                                                                (((S == 1 ? 4 * qd + s : 4 * (g * PER + s) + qd) ^ spread<S>(xrow)) * 16));
            f32x4 start[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                start[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < PER; ++s)
                    start[i] = mfma_bf16(__builtin_bit_cast(bf16x8, minus), fx[s][i], start[i]);
            }
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                f32x4 sum[MT];
                uint32_t codes[PER];
                if constexpr (S == 1) {
                    const u32x4 all = *reinterpret_cast<const u32x4*>(pw + j * 1024);
#pragma unroll
                    for (int s = 0; s < PER; ++s) codes[s] = all[s];
                } else {
#pragma unroll
                    for (int s = 0; s < PER; ++s)
                        codes[s] = *reinterpret_cast<const uint32_t*>(pw + j * 1024 + (g * PER + s) * 256);
                }
#pragma unroll
                for (int s = 0; s < PER; ++s) {
                    const bf16x8 fw = offset_codes(codes[s]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) sum[i] = mfma_bf16(fw, fx[s][i], s == 0 ? start[i] : sum[i]);
                }
                f32x4 scale;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    scale[r] = AHEAD ? all[j * S + (r * S + g) / 4][(r * S + g) % 4] : ps[j * 16 * S + r * S + g];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(scale[r], sum[i][r], acc[i][j][r]);
            }
        }
        cur = cur == RING - 1 ? 0 : cur + 1;
        next = next == RING - 1 ? 0 : next + 1;
    }
    const int cols = strips * 16 < Sh::COLS ? strips * 16 : Sh::COLS;
    const int64_t col0 = static_cast<int64_t>(ct) * Sh::COLS;
    if constexpr (Sh::kJoin) {
        // the parts' sums, in order, through LDS
        constexpr int kSums = 16 * MT * Sh::kSumRow;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NS; ++j)
                *reinterpret_cast<f32x4*>(lds + part * kSums + (i * 16 + i16) * Sh::kSumRow +
                                          ((wave * NS + j) * 16 + 4 * qd) * 4) = acc[i][j];
        __syncthreads();
        for (int e = threadIdx.x; e < t.nrows * (cols / 4); e += Sh::kThreads) {
            const int r = e / (cols / 4), c = (e - r * (cols / 4)) * 4;
            const uint8_t* from = lds + r * Sh::kSumRow + c * 4;
            f32x4 v = *reinterpret_cast<const f32x4*>(from);
#pragma unroll
            for (int p = 1; p < KS; ++p) v += *reinterpret_cast<const f32x4*>(from + p * kSums);
            const int64_t at = (t.row0 + r) * a.N + col0 + c;
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            if (LINEAR) {
                if (a.bias) v += *reinterpret_cast<const f32x4*>(a.bias + col0 + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = act_value(v[i], a.act);
                if (a.residual) {
                    const u32x2 w = *reinterpret_cast<const u32x2*>(a.residual + at);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        v[2 * i] += __uint_as_float(w[i] << 16);
                        v[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
                    }
                }
            }
            if (a.out_fp32) *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = v;
            else
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) =
                    u32x2{pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3])};
        }
    } else {
        store_all<kFwd, LINEAR ? Epilogue::kLinear : Epilogue::kPlain, MT, NS / 2>(
            a, acc, Place{t.row0, a.N, col0, t.nrows, wave * NS * 16, cols}, [&](int i) { return 16 * i; },
            lane);
    }
}

namespace {

template <typename Sh, bool LINEAR, int S>
hipError_t launch(const Int4Args& a, hipStream_t stream) {
    static LdsDevices allowed;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(&int4_kernel<Sh, LINEAR, S>), Sh::lds(S), allowed);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((int4_kernel<Sh, LINEAR, S>), block_grid(matmul_blocks<kFwd, Sh::ROWS, Sh::COLS>(a.m)),
                       dim3(Sh::kThreads), Sh::lds(S), stream, a);
    return hipGetLastError();
}

// the shape is one of int4_rule.h, whose table has its sizes
template <typename Sh>
hipError_t launch_shape(bool linear, int group, const Int4Args& a, hipStream_t stream) {
    switch (group) {
        case 128: return linear ? launch<Sh, true, 1>(a, stream) : launch<Sh, false, 1>(a, stream);
        case 64: return linear ? launch<Sh, true, 2>(a, stream) : launch<Sh, false, 2>(a, stream);
        default: return linear ? launch<Sh, true, 4>(a, stream) : launch<Sh, false, 4>(a, stream);
    }
}

}  // namespace

hipError_t launch_int4(Int4Shape shape, bool linear, int group, const Int4Args& a, hipStream_t stream) {
    switch (shape) {
        case Int4Shape::k4x16p8: return launch_shape<Shape<4, 1, 1, 8, 5>>(linear, group, a, stream);
        case Int4Shape::k4x128p2: return launch_shape<Shape<4, 2, 4, 2, 2>>(linear, group, a, stream);
        case Int4Shape::k16x32p8: return launch_shape<Shape<16, 1, 2, 8, 3>>(linear, group, a, stream);
        case Int4Shape::k16x64p2: return launch_shape<Shape<16, 4, 1, 2, 4>>(linear, group, a, stream);
        case Int4Shape::k16x64p8: return launch_shape<Shape<16, 1, 4, 8, 2>>(linear, group, a, stream);
        case Int4Shape::k16x256: return launch_shape<Shape<16, 4, 4, 1, 2>>(linear, group, a, stream);
        case Int4Shape::k32x64p4: return launch_shape<Shape<32, 2, 2, 4, 2>>(linear, group, a, stream);
        case Int4Shape::k32x128p4: return launch_shape<Shape<32, 2, 4, 4, 2>>(linear, group, a, stream);
        case Int4Shape::k32x256: return launch_shape<Shape<32, 4, 4, 1, 2>>(linear, group, a, stream);
        case Int4Shape::k48x64p4: return launch_shape<Shape<48, 2, 2, 4, 2>>(linear, group, a, stream);
        case Int4Shape::k48x256: return launch_shape<Shape<48, 4, 4, 1, 2>>(linear, group, a, stream);
        case Int4Shape::k64x128: return launch_shape<Shape<64, 4, 2, 1, 2>>(linear, group, a, stream);
        case Int4Shape::k64x256: return launch_shape<Shape<64, 4, 4, 1, 2>>(linear, group, a, stream);
        case Int4Shape::kCount: break;
    }
    return hipErrorInvalidValue;
}

}  // namespace moe
