// matmul.h -- the products of grouped_matmul, its gradients and linear: operands,
// tile lookup, LDS staging and fragment reads shared by the kernels of
// matmul_tile.hip, matmul256.hip, matmul_split.hip and matmul_stream.hip.
//
// One launch computes, for every group e (rows offsets[e] .. offsets[e+1] - 1 of
// the row operands; one group of P rows when offsets is null):
//   kFwd  y[s]  = x[s] W_e^T               out [P, N], reduced over K
//   kDx   dx[s] = dy[s] W_e                out [P, K], reduced over N
//   kDw   dW_e  = sum_s dy[s]^T x[s]       out [E, N, K], reduced over the group's rows
// with x [P, K], dy [P, N] and W [E, N, K] bf16 row-major, accumulated in fp32.
//
// As C[m][n] = sum_r A(m, r) B(n, r), an operand is stored either with r
// contiguous (x and W of kFwd, dy of kDx) or with m / n contiguous (W of kDx, both
// operands of kDw). Both kinds are staged by 16-byte global -> LDS loads whose
// lanes cover whole 128-byte lines, and both are read as MFMA fragments without a
// transposed copy: the first kind by 16-byte reads, the second by the transposing
// 8-byte reads of gfx950 (16 lanes read 4 rows of 16 values and each gets a column).
#pragma once

#include <type_traits>

#include "common.h"
#include "train.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kStepR = 64;  // reduction depth of a staged step

// 16 zero bytes: what a lane loads for a piece past the end of the reduction
static __device__ __constant__ const uint32_t g_zero16[4] __attribute__((aligned(16))) = {0, 0, 0, 0};

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
        (const __attribute__((address_space(3))) void*)p));
}

// 16 bytes per lane from `src` (any lane's address) to LDS at dst + 16 * lane (dst
// uniform over the wave), counted by vmcnt. In assembly because the compiler
// waits for all such loads before any LDS read that it cannot tell apart from
// their target, which would undo the prefetch; the kernels wait for them
// themselves, with wait_loads and a barrier, before the stage is read. The load has no
// destination register. m0 holds the LDS address; a write of it needs one wait
// state before the load.
__device__ __forceinline__ void lds_load16(const void* src, uint32_t dst) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(src), "{m0}"(__builtin_amdgcn_readfirstlane(dst))
                 : "memory");
}
// the same with the source as a uniform base and a 32-bit byte offset
__device__ __forceinline__ void lds_load16(const uint8_t* base, uint32_t off, uint32_t dst) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(base), "{m0}"(__builtin_amdgcn_readfirstlane(dst))
                 : "memory");
}

// Waits until at most N of this wave's loads to LDS are outstanding.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A value that is the same in all lanes, for a scalar register.
__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// ---------------------------------------------------------------- tile lookup

struct MatTile {
    int group;
    int64_t row0;  // first row (kFwd, kDx: of the row operand; kDw: of the group)
    int nrows;     // rows of the tile (kDw: of the group)
};

// Rows of group e, clamped into [0, P]: offsets out of order or out of range give
// wrong or empty groups, never an access outside the operands.
__device__ __forceinline__ void group_rows(const MatmulArgs& a, int e, int64_t& first, int& count) {
    if (!a.offsets) {
        first = 0;
        count = static_cast<int>(a.P);
        return;
    }
    const int P = static_cast<int>(a.P);
    int lo = a.offsets[e], hi = a.offsets[e + 1];
    lo = lo < 0 ? 0 : lo > P ? P : lo;
    hi = hi < lo ? lo : hi > P ? P : hi;
    first = lo;
    count = hi - lo;
}

// The row tiles of all groups, BM rows each, in group order: every wave scans
// the group sizes by itself (four groups a lane, kMaxExperts in all), which needs
// neither LDS nor a table written by an earlier launch.
template <int BM>
struct RowTiles {
    int first[4], count[4], tiles[4];
    int before;  // row tiles of the groups of lower lanes
    int total;

    __device__ __forceinline__ void scan(const MatmulArgs& a, int lane) {
        int sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 4 * lane + i;
            first[i] = count[i] = tiles[i] = 0;
            if (e < a.E) {
                int64_t f;
                group_rows(a, e, f, count[i]);
                first[i] = static_cast<int>(f);
                tiles[i] = (count[i] + BM - 1) / BM;
            }
            sum += tiles[i];
        }
        int incl = sum;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off, kWave);
            if (lane >= off) incl += v;
        }
        before = incl - sum;
        total = __builtin_amdgcn_readlane(incl, 63);
    }

    // row tile rt < total
    __device__ __forceinline__ MatTile find(int rt, int lane) const {
        int local = rt - before, g = -1, f = 0, c = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (g < 0 && local >= 0 && local < tiles[i]) {
                g = 4 * lane + i;
                f = first[i] + local * BM;
                c = count[i] - local * BM;
            }
            if (g < 0) local -= tiles[i];
        }
        const uint64_t hit = __ballot(g >= 0);
        const int src = __builtin_amdgcn_readfirstlane(__ffsll(static_cast<unsigned long long>(hit)) - 1);
        MatTile t;
        t.group = __builtin_amdgcn_readlane(g, src);
        t.row0 = __builtin_amdgcn_readlane(f, src);
        const int left = __builtin_amdgcn_readlane(c, src);
        t.nrows = left < BM ? left : BM;
        return t;
    }
};

// Row tile rt of one group of all rows: nothing to read before the first request (a dense
// 1 x 8192 x 5120: 14.4 against 14.9 us).
template <int BM>
__device__ __forceinline__ MatTile dense_tile(const MatmulArgs& a, int rt) {
    const int64_t row0 = static_cast<int64_t>(rt) * BM, left = a.P - row0;
    return MatTile{0, row0, static_cast<int>(left < BM ? left : BM)};
}

// Block -> tile. Blocks are dealt to the 8 XCDs round robin, and each XCD takes
// a contiguous range of the tiles, so that the tiles it runs at once share operand
// panels in its L2. Inside a range the walk takes BAND row tiles down each column
// of tiles before the next column.
template <int BAND>
__device__ __forceinline__ void band_walk(int64_t lin, int rows, int cols, int& rt, int& ct) {
    const int64_t span = static_cast<int64_t>(BAND) * cols;
    const int band = static_cast<int>(lin / span);
    const int within = static_cast<int>(lin - band * span);
    const int here = rows - band * BAND < BAND ? rows - band * BAND : BAND;
    rt = band * BAND + within % here;
    ct = within / here;
}

// The tile of this block; false: none. kDw: every group has the same tiles. Where they
// are many, each XCD takes a contiguous eighth of each group's, so that groups of
// unequal length weigh equally on all; else it takes an eighth of all groups' tiles.
constexpr int64_t kManyTiles = 64;
template <int MODE, int BM, int BN, int BAND>
__device__ __forceinline__ bool find_tile(const MatmulArgs& a, int lane, MatTile& t, int& rt, int& ct) {
    const int ncol = static_cast<int>(((MODE == kFwd ? a.N : a.K) + BN - 1) / BN);
    const int xcd = blockIdx.x & 7;
    // a grid of several rows has kGridX blocks in each
    int64_t lin = (blockIdx.x >> 3) + blockIdx.y * (kGridX >> 3);
    if (MODE == kDw) {
        const int nrow = static_cast<int>((a.N + BM - 1) / BM);
        const int64_t n = static_cast<int64_t>(nrow) * ncol;
        const int64_t all = n < kManyTiles ? n * a.E : n;
        const int64_t first = all * xcd / 8, mine = all * (xcd + 1) / 8 - first;
        if (lin >= (n < kManyTiles ? mine : mine * a.E)) return false;
        if (n < kManyTiles) {
            t.group = static_cast<int>((first + lin) / n);
            lin = first + lin - t.group * n;
        } else {
            t.group = static_cast<int>(lin / mine);
            lin = first + lin - t.group * mine;
        }
        band_walk<BAND>(lin, nrow, ncol, rt, ct);
        group_rows(a, t.group, t.row0, t.nrows);
        return !(a.accumulate && t.nrows == 0);
    }
    RowTiles<BM> tiles;
    if (a.offsets) tiles.scan(a, lane);
    else tiles.total = static_cast<int>((a.P + BM - 1) / BM);
    const int64_t n = static_cast<int64_t>(tiles.total) * ncol;
    const int64_t first = n * xcd / 8, mine = n * (xcd + 1) / 8 - first;
    if (lin >= mine) return false;
    band_walk<BAND>(first + lin, tiles.total, ncol, rt, ct);
    t = a.offsets ? tiles.find(rt, lane) : dense_tile<BM>(a, rt);
    return true;
}

// Blocks of a launch, an upper bound: the host does not know the group sizes.
template <int MODE, int BM, int BN>
inline int64_t matmul_blocks(const MatmulArgs& a) {
    const int64_t ncol = ((MODE == kFwd ? a.N : a.K) + BN - 1) / BN;
    int64_t mine;  // the most tiles of an XCD
    if (MODE == kDw) {
        const int64_t n = ((a.N + BM - 1) / BM) * ncol;
        mine = n < kManyTiles ? (a.E * n + 7) / 8 : a.E * ((n + 7) / 8);
    } else {
        // row tiles: full ones and at most one partial tile for each group with rows
        const int64_t partial = a.E < a.P ? a.E : a.P;
        mine = ((a.P / BM + partial) * ncol + 7) / 8;
    }
    return 8 * mine;
}

// ------------------------------------------------------------------- staging

// LDS order of a tile stored with r contiguous, rows of 64 values: row-major, 128
// bytes a row, its eight 16-byte pieces XORed by row_spread. A 16-byte read is
// served 16 lanes at a time over 64 banks (the lanes sharing lane bit 5 and
// the parity of bits 2..4); reading 16 rows in a row, the 16 touch 16 different
// groups of four banks.
__device__ __forceinline__ int row_spread(int r) { return (r >> 1) & 7; }

// LDS order of a tile stored with m / n contiguous, 64 rows of r x SIZE values:
// row-major, 2 SIZE bytes a row, its 16-byte pieces XORed by red_spread. A transposing
// 8-byte read is served 32 lanes at a time: 8 rows (four in a row, twice, 8 apart)
// of 32 bytes each, which the even XOR values put on 16 different groups of four banks
// (with rows of 128 and 64 bytes the lowest bits of the row do their part).
template <int SIZE>
__device__ __forceinline__ int red_spread(int r) {
    if (SIZE == 32) return ((r >> 3) & 1) << 1;
    if (SIZE == 64) return (((r >> 3) & 1) << 2) | (r & 2);
    return (((r >> 3) & 1) << 3) | ((r & 3) << 1);
}

// Tile row i of a gated block's weights: 16 gate rows, then the 16 up rows of the same
// outputs, and so on, so that a wave's neighbouring sub-tiles are the two factors of a
// product and meet in one lane's registers. `valid`: rows of both in the tile.
__device__ __forceinline__ int64_t gated_row(int i, int valid, int64_t apart) {
    const int out = (i >> 5) * 16 + (i & 15), last = (valid >> 1) - 1;
    return (out < last ? out : last) + ((i >> 4) & 1) * apart;
}

// Global -> LDS staging of one operand's tile, 1 KB a wave and load.
// TR: m / n contiguous.
template <bool TR, int SIZE, int WAVES>
struct Stager {
    static constexpr int kLoads = SIZE / 8 / WAVES;  // per wave and step
    static constexpr int kPieces = TR ? SIZE / 8 : 8;  // 16-byte pieces a tile row
    static constexpr int kRows = 64 / kPieces;         // tile rows a load
    const uint8_t* base;      // uniform: the tile's first value at step 0
    int64_t step;             // bytes from step to step
    uint32_t off[kLoads];     // this lane's source, relative to base
    int wave, lane;

    // TR = false: tile row i is row i of `p` (ld values apart), rows past `valid`
    // repeat the last one. TR = true: tile row i is row i of the reduction, values
    // past `valid` (a multiple of 8) repeat the last piece. What they give is dropped.
    // GATED: tile rows are those of two matrices `apart` rows apart, by turns (gated_row).
    template <bool GATED = false>
    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int valid, int wave_, int lane_,
                                         int64_t apart = 0) {
        wave = wave_;
        lane = lane_;
        base = reinterpret_cast<const uint8_t*>(uniform(reinterpret_cast<uint64_t>(p)));
        step = TR ? kStepR * ld * 2 : kStepR * 2;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = tile_row(i);
            if (TR) {
                int c = piece(i) * 8;
                c = c < valid ? c : valid - 8;
                off[i] = static_cast<uint32_t>((r * ld + c) * 2);
            } else {
                const int64_t m = GATED ? gated_row(r, valid, apart) : r < valid ? r : valid - 1;
                off[i] = static_cast<uint32_t>((m * ld + piece(i) * 8) * 2);
            }
        }
    }
    __device__ __forceinline__ int tile_row(int i) const {
        return (wave + i * WAVES) * kRows + lane / kPieces;
    }
    // the 16-byte piece of its row that this lane loads
    __device__ __forceinline__ int piece(int i) const {
        const int r = tile_row(i);
        return (lane % kPieces) ^ (TR ? red_spread<SIZE>(r) : row_spread(r));
    }
    // loads [FROM, TO) of step k into the tile at LDS address `lds`; `red`: length of
    // the reduction
    template <int FROM = 0, int TO = kLoads>
    __device__ __forceinline__ void load(uint32_t lds, int k, int64_t red) const {
        const uint8_t* b = base + k * step;
        const int64_t left = red - static_cast<int64_t>(k) * kStepR;
        if (left >= kStepR) {
#pragma unroll
            for (int i = FROM; i < TO; ++i) lds_load16(b, off[i], lds + (wave + i * WAVES) * 1024);
        } else {
#pragma unroll
            for (int i = FROM; i < TO; ++i) {
                const int at = TR ? tile_row(i) : piece(i) * 8;
                const void* src = at < left ? static_cast<const void*>(b + off[i])
                                            : static_cast<const void*>(g_zero16);
                lds_load16(src, lds + (wave + i * WAVES) * 1024);
            }
        }
    }
};

// ---------------------------------------------------------------- fragments
//
// v_mfma_f32_16x16x32_bf16: lane l holds row l % 16, values 8 (l / 16) .. + 7 of
// the 32-deep slice. B is passed first, so that D's rows are B's: lane l gets
// D[4 (l / 16) + i][l % 16], i.e. four consecutive columns of the output in one row.

// Reader of one operand's fragments from a tile of SIZE values of m / n.
template <bool TR, int SIZE>
struct Reader {
    static constexpr int kSubs = SIZE < 128 ? 2 : 4;
    int at[TR ? kSubs : 2];  // byte address, TR: by sub-tile, else by slice s

    // row0: the wave's first row (m or n) in the tile, a multiple of 32
    __device__ __forceinline__ void init(int row0, int lane) {
        const int i16 = lane & 15, q = lane >> 4;
        if (TR) {
            // lane 4 j + c of a 16-lane group reads row 8 q + j (and + 4), values 4c .. 4c + 3
            const int row = 8 * q + (i16 >> 2), c = i16 & 3;
#pragma unroll
            for (int i = 0; i < kSubs; ++i)
                at[i] = row * SIZE * 2 + (((row0 / 8 + 2 * i + (c >> 1)) ^ red_spread<SIZE>(row)) * 16) + (c & 1) * 8;
        } else {
            const int r = row0 + i16;
#pragma unroll
            for (int s = 0; s < 2; ++s) at[s] = r * 128 + (((4 * s + q) ^ row_spread(r)) * 16);
        }
    }
    // fragment of sub-tile i (rows row0 + 16 i ..; i < 4), slice s
    __device__ __forceinline__ bf16x8 read(const uint8_t* lds, int i, int s) const {
        if (TR) {
            const uint8_t* p = lds + s * 32 * SIZE * 2 + at[i];
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(p));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(p + 4 * SIZE * 2));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return *reinterpret_cast<const bf16x8*>(lds + at[s] + i * 16 * 128);
    }
};

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 b, bf16x8 a, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}

// ------------------------------------------------------------------ epilogue

__device__ __forceinline__ u32x4 pack8(const float* v) {
    return u32x4{pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]),
                 pack_bf16x2_rn(v[6], v[7])};
}
__device__ __forceinline__ void unpack8(u32x4 w, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Two neighbouring sub-tiles' four columns a lane -> eight consecutive columns:
// lane groups q and q ^ 1 exchange halves, after which group q holds the columns
// 16 (q % 2) + 8 (q / 2) .. + 7 of the pair's 32.
__device__ __forceinline__ void eight_columns(f32x4 x, f32x4 y, float* v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[r]), __float_as_uint(y[r]), false, false);
        v[r] = __uint_as_float(p[0]);
        v[4 + r] = __uint_as_float(p[1]);
    }
}
__device__ __forceinline__ int eight_columns_at(int q) { return 16 * (q & 1) + 8 * (q >> 1); }

// Rows of the output start on 128-byte lines, so that stores of whole tiles write whole lines.
__device__ __forceinline__ bool whole_lines(const MatmulArgs& a, int64_t ld) {
    return ((reinterpret_cast<uintptr_t>(a.out) | static_cast<uintptr_t>(ld * (a.out_fp32 ? 4 : 2))) & 127) == 0;
}

// Where a wave's accumulators go: 16 rows from row0(i) for sub-tile row i, 32 columns from
// col0 for each pair of sub-tiles; rows and columns of the tile end at rows and cols,
// which stands at out_row, out_col of the output.
struct Place {
    int64_t out_row, ld, out_col;
    int rows, col0, cols;
};

// The products' own results of NI x 16 rows, 32 JJ columns. Lanes l and l ^ 8 exchange
// halves, so that a store instruction covers whole 128-byte lines: 8 rows of 64 bf16
// or 32 fp32 values. (Without: 64-byte pieces. 128 x 1000 x 712 weight gradients in
// fp32 116 us, 95 with.) STREAM: the lines are not kept in L2; a weight gradient is read
// much later, and its lines would push the operands out (32 x 4096 x 4096: 360 us, 306
// with), but parts of lines must meet there. ACC: added to the old values, which are
// loaded for two sub-tile rows at once.
template <int NI, int JJ, bool STREAM, bool ACC, typename Row>
__device__ __forceinline__ void store_rows(const MatmulArgs& a, const f32x4 (*acc)[2 * JJ], const Place& at,
                                           Row&& row0, int lane) {
    const int i16 = lane & 15, q = lane >> 4;
    const bool low = i16 < 8;
    const int size = a.out_fp32 ? 4 : 2;
    // the value of lane l ^ 8 (a rotation by 8 in each row of 16 lanes)
    auto other = [](uint32_t v) {
        return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x128, 0xf, 0xf, true));
    };
    constexpr int BATCH = ACC ? 2 : 1;
#pragma unroll
    for (int i0 = 0; i0 < NI; i0 += BATCH) {
        u32x4 v[BATCH][JJ][2];
        uint8_t* p[BATCH][JJ][2];
        bool ok[BATCH][JJ][2];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int row = row0(i0 + b);  // negative: none
            // first: rows 0..7, second: 8..15; low lanes the first half line, high lanes the second
            auto put = [&](int n, const u32x4& first, const u32x4& second, int col, int half, int width)
                           __attribute__((always_inline)) {
                u32x4 got;
#pragma unroll
                for (int k = 0; k < 4; ++k) got[k] = other(low ? second[k] : first[k]);
                v[b][n][0] = low ? first : got;
                v[b][n][1] = low ? got : second;
                const int c = col + (low ? 0 : half), r = row + (i16 & 7);
                p[b][n][0] = static_cast<uint8_t*>(a.out) + ((at.out_row + r) * at.ld + at.out_col + c) * size;
                p[b][n][1] = p[b][n][0] + 8 * at.ld * size;
                ok[b][n][0] = row >= 0 && r < at.rows && c + width <= at.cols;
                ok[b][n][1] = row >= 0 && r + 8 < at.rows && c + width <= at.cols;
            };
            const f32x4* x = acc[i0 + b];
            if (a.out_fp32) {
#pragma unroll
                for (int h = 0; h < JJ; ++h)
                    put(h, __builtin_bit_cast(u32x4, x[2 * h]), __builtin_bit_cast(u32x4, x[2 * h + 1]),
                        at.col0 + 32 * h + 4 * q, 16, 4);
            } else {
#pragma unroll
                for (int h = 0; h < JJ; h += 2) {
                    float lo[8], hi[8];
                    eight_columns(x[2 * h], x[2 * h + 1], lo);
                    if (JJ > 1) eight_columns(x[JJ > 1 ? 2 * h + 2 : 0], x[JJ > 1 ? 2 * h + 3 : 0], hi);
                    if (JJ > 1) {
                        put(h, pack8(lo), pack8(hi), at.col0 + 32 * h + eight_columns_at(q), 32, 8);
                        ok[b][h + JJ / 2][0] = ok[b][h + JJ / 2][1] = false;
                    } else {
                        // 32 columns: no second half line to exchange
                        const int c = at.col0 + eight_columns_at(q), r = row + i16;
                        v[b][0][0] = pack8(lo);
                        p[b][0][0] = static_cast<uint8_t*>(a.out) + ((at.out_row + r) * at.ld + at.out_col + c) * size;
                        ok[b][0][0] = row >= 0 && r < at.rows && c + 8 <= at.cols;
                        ok[b][0][1] = false;
                    }
                }
            }
        }
        if (ACC) {
            u32x4 old[BATCH][JJ][2];
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int n = 0; n < JJ; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (ok[b][n][k]) old[b][n][k] = *reinterpret_cast<const u32x4*>(p[b][n][k]);
#pragma unroll
            for (int b = 0; b < BATCH; ++b)
#pragma unroll
                for (int n = 0; n < JJ; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (!ok[b][n][k]) continue;
                        v[b][n][k] = __builtin_bit_cast(
                            u32x4, __builtin_bit_cast(f32x4, v[b][n][k]) + __builtin_bit_cast(f32x4, old[b][n][k]));
                    }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int n = 0; n < JJ; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (!ok[b][n][k]) continue;
                    u32x4* to = reinterpret_cast<u32x4*>(p[b][n][k]);
                    if (STREAM) __builtin_nontemporal_store(v[b][n][k], to);
                    else *to = v[b][n][k];
                }
    }
}

// Results with something to be added or applied: for linear, bias, activation and
// residual; else the old values (accumulate). One rounding at the end. The bias is
// loaded once, the residual or old values for two sub-tile rows at once before any
// is stored: one at a time, each would wait for its own load (14203 x 4568 x 488 with
// bias, gelu and residual: 178 us, 158 with).
// ACT is a template argument: the switch would be taken, and its code repeated, for every
// value.
template <bool LINEAR, int ACT, int NI, int JJ, typename Row>
__device__ __forceinline__ void store_applied(const MatmulArgs& a, const f32x4 (*acc)[2 * JJ], const Place& at,
                                              Row&& row0, int lane) {
    const int i16 = lane & 15, q = lane >> 4;
    constexpr int BATCH = 2;
    float bias[JJ][8];
#pragma unroll
    for (int h = 0; h < JJ; ++h) {
        const int c = at.col0 + 32 * h + eight_columns_at(q);
#pragma unroll
        for (int k = 0; k < 8; ++k) bias[h][k] = 0.f;
        if (LINEAR && a.bias && c < at.cols) {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(a.bias + at.out_col + c);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(a.bias + at.out_col + c + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bias[h][k] = lo[k];
                bias[h][4 + k] = hi[k];
            }
        }
    }
    const uint16_t* add16 = LINEAR ? a.residual
                                   : !a.out_fp32 ? static_cast<const uint16_t*>(a.out) : nullptr;
    const float* add32 = !LINEAR && a.out_fp32 ? static_cast<const float*>(a.out) : nullptr;
#pragma unroll
    for (int i0 = 0; i0 < NI; i0 += BATCH) {
        u32x4 old[BATCH][JJ][LINEAR ? 1 : 2];
        bool ok[BATCH][JJ];
        int64_t pos[BATCH][JJ];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int r0 = row0(i0 + b), r = r0 + i16;
#pragma unroll
            for (int h = 0; h < JJ; ++h) {
                const int c = at.col0 + 32 * h + eight_columns_at(q);
                ok[b][h] = r0 >= 0 && r < at.rows && c < at.cols;
                pos[b][h] = (at.out_row + r) * at.ld + at.out_col + c;
                if (!ok[b][h]) continue;
                if (add16) old[b][h][0] = *reinterpret_cast<const u32x4*>(add16 + pos[b][h]);
                if (!LINEAR && add32) {
                    old[b][h][0] = *reinterpret_cast<const u32x4*>(add32 + pos[b][h]);
                    old[b][h][LINEAR ? 0 : 1] = *reinterpret_cast<const u32x4*>(add32 + pos[b][h] + 4);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int h = 0; h < JJ; ++h) {
                float v[8];
                eight_columns(acc[i0 + b][2 * h], acc[i0 + b][2 * h + 1], v);
                if (!ok[b][h]) continue;
                if (LINEAR) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] += bias[h][k];
                    if (a.z) *reinterpret_cast<u32x4*>(a.z + pos[b][h]) = pack8(v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = act_value(v[k], ACT);
                }
                if (add16) {
                    float r[8];
                    unpack8(old[b][h][0], r);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] += r[k];
                }
                if (!LINEAR && add32) {
                    const f32x4 lo = __builtin_bit_cast(f32x4, old[b][h][0]);
                    const f32x4 hi = __builtin_bit_cast(f32x4, old[b][h][LINEAR ? 0 : 1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        v[k] += lo[k];
                        v[4 + k] += hi[k];
                    }
                }
                if (a.out_fp32) {
                    float* o = static_cast<float*>(a.out) + pos[b][h];
                    *reinterpret_cast<f32x4*>(o) = f32x4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<f32x4*>(o + 4) = f32x4{v[4], v[5], v[6], v[7]};
                } else {
                    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + pos[b][h]) = pack8(v);
                }
            }
    }
}

// N values to bf16, N 8 or 4
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float* v) {
    typedef uint32_t words __attribute__((ext_vector_type(N / 2)));
    words w;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<words*>(p) = w;
}

// A gated block's outputs from sub-tiles that are gate and up by turns: each two give 16
// columns of act(g) u. A pair of them (JJ = 2) goes out eight columns a lane, as above, a
// single one four. z takes g and u as they were before the activation, rounded. 8192 rows over 16
// groups, h = 8192, d = 5120: 1201 us, with z 1245; the product of the same sizes takes 1217 and the
// activation after it 68. A single row 29 us (5.8 TB/s).
template <int ACT, int NI, int JJ, typename Row>
__device__ __forceinline__ void store_gated(const MatmulArgs& a, const f32x4 (*acc)[2 * JJ], const Place& at,
                                            Row&& row0, int lane) {
    constexpr int W = 4 * JJ;  // columns a lane
    const int i16 = lane & 15, q = lane >> 4;
    const int64_t h = a.N / 2;
    const int c = at.col0 / 2 + (JJ == 2 ? eight_columns_at(q) : 4 * q);
    const int64_t col = at.out_col / 2 + c;
    const bool inside = c < at.cols / 2;
    float bg[W], bu[W];
#pragma unroll
    for (int k = 0; k < W; ++k) bg[k] = bu[k] = 0.f;
    if (a.bias && inside) {
#pragma unroll
        for (int k = 0; k < W; k += 4) {
            *reinterpret_cast<f32x4*>(bg + k) = *reinterpret_cast<const f32x4*>(a.bias + col + k);
            *reinterpret_cast<f32x4*>(bu + k) = *reinterpret_cast<const f32x4*>(a.bias + h + col + k);
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        float g[W], u[W];
        if constexpr (JJ == 2) {
            eight_columns(acc[i][0], acc[i][2], g);
            eight_columns(acc[i][1], acc[i][3], u);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                g[k] = acc[i][0][k];
                u[k] = acc[i][1][k];
            }
        }
        const int r0 = row0(i), r = r0 + i16;
        if (r0 < 0 || r >= at.rows || !inside) continue;
        const int64_t row = at.out_row + r;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            g[k] += bg[k];
            u[k] += bu[k];
        }
        if (a.z) {
            store_bf16<W>(a.z + row * a.N + col, g);
            store_bf16<W>(a.z + row * a.N + h + col, u);
        }
#pragma unroll
        for (int k = 0; k < W; ++k) g[k] = act_value(g[k], ACT) * u[k];
        store_bf16<W>(static_cast<uint16_t*>(a.out) + row * h + col, g);
    }
}

// The gradient of a gated block's projections, from that of its outputs (the products):
// dz = [dh u act'(g) | dh act(g)], and act(g) u where it is wanted. g and u are loaded for two
// sub-tile rows at once, ahead of the stores. Each place of dz is written by the lane
// that read it of z, so that they may be one buffer. At the sizes above 750 us (800 on the slowest of four boxes), against 646 for
// the product and 183 for the two passes after it: bound by the product, and then by the
// 0.67 GB that all blocks move at once as their tiles end.
template <int ACT, int NI, int JJ, typename Row>
__device__ __forceinline__ void store_gated_dz(const MatmulArgs& a, const f32x4 (*acc)[2 * JJ], const Place& at,
                                               Row&& row0, int lane) {
    constexpr int BATCH = 2;
    const int i16 = lane & 15, q = lane >> 4;
    const int64_t h = a.K;
    uint16_t* dz = static_cast<uint16_t*>(a.out);
#pragma unroll
    for (int i0 = 0; i0 < NI; i0 += BATCH) {
        u32x4 z[BATCH][JJ][2];
        bool ok[BATCH][JJ];
        int64_t row[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int r0 = row0(i0 + b), r = r0 + i16;
            row[b] = at.out_row + r;
#pragma unroll
            for (int j = 0; j < JJ; ++j) {
                const int c = at.col0 + 32 * j + eight_columns_at(q);
                ok[b][j] = r0 >= 0 && r < at.rows && c < at.cols;
                if (!ok[b][j]) continue;
                const uint16_t* p = a.gate_z + row[b] * 2 * h + at.out_col + c;
                z[b][j][0] = *reinterpret_cast<const u32x4*>(p);
                z[b][j][1] = *reinterpret_cast<const u32x4*>(p + h);
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int j = 0; j < JJ; ++j) {
                float d[8], g[8], u[8];
                eight_columns(acc[i0 + b][2 * j], acc[i0 + b][2 * j + 1], d);
                if (!ok[b][j]) continue;
                unpack8(z[b][j][0], g);
                unpack8(z[b][j][1], u);
                const int64_t col = at.out_col + at.col0 + 32 * j + eight_columns_at(q);
                float dg[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float v = act_value(g[k], ACT);
                    dg[k] = d[k] * u[k] * act_slope(g[k], ACT);
                    d[k] *= v;
                    u[k] *= v;
                }
                store_bf16<8>(dz + row[b] * 2 * h + col, dg);
                store_bf16<8>(dz + row[b] * 2 * h + h + col, d);
                if (a.gate_y) store_bf16<8>(a.gate_y + row[b] * h + col, u);
            }
    }
}

template <Epilogue EPI, int ACT, int NI, int JJ, typename Row>
__device__ __forceinline__ void store_gated_any(const MatmulArgs& a, const f32x4 (*acc)[2 * JJ], const Place& at,
                                                Row&& row0, int lane) {
    if constexpr (EPI == Epilogue::kGated) store_gated<ACT, NI, JJ>(a, acc, at, row0, lane);
    else store_gated_dz<ACT, NI, JJ>(a, acc, at, row0, lane);
}

// All of a wave's results.
template <int MODE, Epilogue EPI, int NI, int JJ, typename Row>
__device__ __forceinline__ void store_all(const MatmulArgs& a, const f32x4 (*acc)[2 * JJ], const Place& at,
                                          Row&& row0, int lane) {
    if constexpr (EPI == Epilogue::kGated || EPI == Epilogue::kGatedDz) {
        // the activation as a compile-time constant, as below
        switch (a.act) {
            case MOE_ACT_RELU: return store_gated_any<EPI, MOE_ACT_RELU, NI, JJ>(a, acc, at, row0, lane);
            case MOE_ACT_SILU: return store_gated_any<EPI, MOE_ACT_SILU, NI, JJ>(a, acc, at, row0, lane);
            case MOE_ACT_GELU: return store_gated_any<EPI, MOE_ACT_GELU, NI, JJ>(a, acc, at, row0, lane);
            case MOE_ACT_GELU_TANH: return store_gated_any<EPI, MOE_ACT_GELU_TANH, NI, JJ>(a, acc, at, row0, lane);
            default: return store_gated_any<EPI, MOE_ACT_NONE, NI, JJ>(a, acc, at, row0, lane);
        }
    }
    constexpr bool LINEAR = EPI == Epilogue::kLinear;
    if (LINEAR && (a.bias || a.z || a.residual || a.act != MOE_ACT_NONE)) {
        switch (a.act) {
            case MOE_ACT_RELU: return store_applied<true, MOE_ACT_RELU, NI, JJ>(a, acc, at, row0, lane);
            case MOE_ACT_SILU: return store_applied<true, MOE_ACT_SILU, NI, JJ>(a, acc, at, row0, lane);
            case MOE_ACT_GELU: return store_applied<true, MOE_ACT_GELU, NI, JJ>(a, acc, at, row0, lane);
            case MOE_ACT_GELU_TANH: return store_applied<true, MOE_ACT_GELU_TANH, NI, JJ>(a, acc, at, row0, lane);
            default: return store_applied<true, MOE_ACT_NONE, NI, JJ>(a, acc, at, row0, lane);
        }
    } else if (MODE == kDw && a.accumulate) {
        if (a.out_fp32) store_rows<NI, JJ, false, true>(a, acc, at, row0, lane);
        else store_applied<false, MOE_ACT_NONE, NI, JJ>(a, acc, at, row0, lane);
    } else if (MODE == kDw && whole_lines(a, at.ld)) {
        store_rows<NI, JJ, true, false>(a, acc, at, row0, lane);
    } else {
        store_rows<NI, JJ, false, false>(a, acc, at, row0, lane);
    }
}

// One value of a linear layer or product.
template <bool LINEAR>
__device__ __forceinline__ void store1(const MatmulArgs& a, int64_t row, int64_t ld, int64_t col, float v) {
    const int64_t at = row * ld + col;
    if (LINEAR) {
        if (a.bias) v += a.bias[col];
        if (a.z) a.z[at] = static_cast<uint16_t>(pack_bf16x2_rn(v, 0.f));
        v = act_value(v, a.act);
        if (a.residual) v += bf16_to_f32(a.residual[at]);
    }
    if (a.out_fp32) static_cast<float*>(a.out)[at] = v;
    else static_cast<uint16_t*>(a.out)[at] = static_cast<uint16_t>(pack_bf16x2_rn(v, 0.f));
}

// One output of a gated block from its two factors.
__device__ __forceinline__ void store1_gated(const MatmulArgs& a, int64_t row, int64_t col, float g, float u) {
    const int64_t h = a.N / 2;
    if (a.bias) {
        g += a.bias[col];
        u += a.bias[h + col];
    }
    if (a.z) {
        a.z[row * a.N + col] = static_cast<uint16_t>(pack_bf16x2_rn(g, 0.f));
        a.z[row * a.N + h + col] = static_cast<uint16_t>(pack_bf16x2_rn(u, 0.f));
    }
    static_cast<uint16_t*>(a.out)[row * h + col] =
        static_cast<uint16_t>(pack_bf16x2_rn(act_value(g, a.act) * u, 0.f));
}

// calls `f` with a launch's direction and epilogue as compile-time constants
template <typename F>
inline hipError_t with_mode(int mode, Epilogue e, F&& f) {
    using std::integral_constant;
    if (mode == kDw) return f(integral_constant<int, kDw>{}, integral_constant<Epilogue, Epilogue::kPlain>{});
    if (mode == kDx) {
        if (e == Epilogue::kGatedDz)
            return f(integral_constant<int, kDx>{}, integral_constant<Epilogue, Epilogue::kGatedDz>{});
        return f(integral_constant<int, kDx>{}, integral_constant<Epilogue, Epilogue::kPlain>{});
    }
    if (e == Epilogue::kGated) return f(integral_constant<int, kFwd>{}, integral_constant<Epilogue, Epilogue::kGated>{});
    if (e == Epilogue::kLinear) return f(integral_constant<int, kFwd>{}, integral_constant<Epilogue, Epilogue::kLinear>{});
    return f(integral_constant<int, kFwd>{}, integral_constant<Epilogue, Epilogue::kPlain>{});
}

// The operands of one tile as C[m][n] = sum_r A(m, r) B(n, r).
template <int MODE>
struct Operands {
    const uint16_t *a, *b;  // at the tile's first row / column
    int64_t lda, ldb;
    int64_t red;            // length of the reduction
    int rows, cols;         // valid rows and columns of the tile, from its origin
    int64_t out_row, ldo, col0;
};

// part: 0 or 1 for the first or last BM / 2 rows of the tile, -1 for all; `rows` is not
// positive for a half that has none. A gated block's columns are rows of both its matrices, b
// at the first of its gate rows.
template <int MODE, int BM, int BN, Epilogue EPI>
__device__ __forceinline__ Operands<MODE> operands(const MatmulArgs& a, const MatTile& t, int rt, int ct,
                                                   int part) {
    const int skip = part > 0 ? BM / 2 : 0, most = part < 0 ? BM : BM / 2;
    Operands<MODE> o;
    o.col0 = static_cast<int64_t>(ct) * BN;
    const int64_t ncols = (MODE == kFwd ? a.N : a.K) - o.col0;
    o.cols = static_cast<int>(ncols < BN ? ncols : BN);
    if (MODE == kDw) {
        const int64_t m0 = static_cast<int64_t>(rt) * BM + skip;
        o.a = a.a + t.row0 * a.N + m0;
        o.b = a.b + t.row0 * a.K + o.col0;
        o.lda = a.N;
        o.ldb = a.K;
        o.red = t.nrows;
        const int64_t nr = a.N - m0;
        o.rows = static_cast<int>(nr < most ? nr : most);
        o.out_row = t.group * a.N + m0;
        o.ldo = a.K;
    } else {
        const int64_t kd = MODE == kFwd ? a.K : a.N;
        const uint16_t* w = a.b + static_cast<int64_t>(t.group) * a.N * a.K;
        const int64_t row0 = t.row0 + skip;
        o.a = a.a + row0 * kd;
        o.b = MODE == kFwd ? w + (EPI == Epilogue::kGated ? o.col0 / 2 : o.col0) * a.K : w + o.col0;
        o.lda = kd;
        o.ldb = a.K;
        o.red = kd;
        o.rows = t.nrows - skip < most ? t.nrows - skip : most;
        o.out_row = row0;
        o.ldo = MODE == kFwd ? a.N : a.K;
    }
    return o;
}

}  // namespace moe
