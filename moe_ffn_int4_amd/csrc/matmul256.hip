// matmul256.hip -- the products of matmul.h in 256 x 256 tiles, for groups of
// hundreds of rows.
//
// One block of 8 waves a CU, in a 2 x 4 grid of 128 x 64 wave tiles (8 x 4 products
// of 16 x 16 x 32, 128 accumulators a lane, two waves a SIMD). The reduction runs in
// 64-deep steps through LDS, an operand's tile of a step in two halves of 16 KB:
// A0 / A1 the first / last 64 rows of every wave's 128, B0 / B1 the first / last 32
// columns of every wave's 64. A step is two phases of 32 products a wave:
//     phase 0: read A0, B0 and B1, multiply A0 by both
//     phase 1: read A1, multiply it by both
// over two stages; each phase requests what its predecessor has just finished
// reading, for a later step, so that three phases (about 3000 cycles) lie between most
// requests and their use, and no wait is for the youngest request.
//
// The four waves 4..7 run half a phase behind 0..3 (they take one more barrier
// at the start): while the one wave of a SIMD reads fragments, the other multiplies,
// and the LDS reads and requests of a phase pass under the 512 cycles of the other
// half's products. (A step in four phases of 16 products was slower: the reads' latency
// and the barriers then outlast the 256 cycles of products. 4096 x 4096 x 4096 dense:
// 109 against 97 us; now at 1420 TFLOP/s, where the clock falls to about 1.9 GHz.)
//
// A tile of at most 128 rows (the end of a group, or half a tile, see find) has waves of
// at most 64 x 64: phase 0 alone, over three stages without A1. The last half of a
// tile's rows is multiplied in as many sub-tiles of 16 as hold rows.
//
// Why each access is safe, in half-phases t (waves 0..3 read at t = 2p and
// multiply at 2p + 1, waves 4..7 one later), a barrier between t and t + 1:
//  * a wave ends its reading half-phase with its own reads done and with all its
//    requests landed that phase p + 1 will read; waves 0..3 do so at the end of t = 2p,
//    waves 4..7 at the end of 2p + 1, and they are first read at t = 2p + 2.
//  * phase p overwrites what phase p - 1 read, at t = 2p the earliest; the last reads
//    of phase p - 1 ended before the barrier after t = 2p - 1.
#include "matmul.h"

namespace moe {

namespace {
constexpr int BM = 256;
constexpr int BN = 256;
constexpr int kWaves = 8;
constexpr int kHalf = 128 * kStepR * 2;  // 16 KB
constexpr int kStages = 9 * kHalf;       // 144 KB: two stages of four halves, or three of three
constexpr int kBand = 4;
constexpr int kXcdCus = 32;

__device__ __forceinline__ void block_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The tiles of this block's XCD, group by group: of each group some of its tiles of 256
// rows, walked in bands of up to kBand rows, then some of its last row of tiles where
// that has at most 128 rows.
//
// XCDs share every group: XCD x takes the contiguous eighth (x + e) % 8 of group e's
// tiles of each kind, so that every XCD has the same work whatever the group sizes (a
// line of all groups' tiles cut by estimated cost: 16 experts, 8192 rows, 16384 x 5120,
// forward 1406 against 1305 us, dx 1428 against 1405). Groups of few tiles would leave
// an XCD one or two of each, with little to share in its L2; their tiles stand in one
// line, of which each XCD takes an eighth: 32 experts of 128 rows, 4096 x 4096 (16 tiles
// each), 224 against 266 us.
struct Group {
    int before, tiles;  // tiles of earlier groups, and of this one, on this XCD
    int whole, start;   // of these, tiles of 256 rows, from the group's tile `start`;
    int column;         // the rest are the small ones from this column
    int first, count;   // rows
};
constexpr int kTable = kMaxExperts * static_cast<int>(sizeof(Group));
constexpr uint32_t kFewTiles = 32;

// first of eighth x of n (the host refuses more than 2^30 tiles)
__device__ __forceinline__ int eighth(uint32_t n, int x) { return static_cast<int>((n >> 3) * x + ((n & 7) * x >> 3)); }

// tiles of BM rows, and whether a smaller one follows them
template <int MODE>
__device__ __forceinline__ void row_tiles(const MatmulArgs& a, int count, int& whole, int& small) {
    if (MODE == kDw) {
        whole = static_cast<int>((a.N + BM - 1) / BM);
        small = 0;
    } else {
        small = count % BM > 0 && count % BM <= BM / 2;
        whole = (count + BM - 1) / BM - small;
    }
}

__device__ __forceinline__ uint32_t inclusive_scan(uint32_t v, int lane) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t u = __shfl_up(v, off, kWave);
        if (lane >= off) v += u;
    }
    return v;
}

// Fills the table (every wave the same values) and returns the number of tiles.
template <int MODE>
__device__ __forceinline__ int fill_table(const MatmulArgs& a, Group* table, int ncol, int lane) {
    const int xcd = blockIdx.x & 7;
    Group g[4];
    int whole[4], small[4];
    uint32_t mine = 0, groups = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * lane + i;
        g[i] = Group{0, 0, 0, 0, 0, 0, 0};
        whole[i] = small[i] = 0;
        if (e < a.E) {
            int64_t first;
            group_rows(a, e, first, g[i].count);
            g[i].first = static_cast<int>(first);
            int w, s;
            row_tiles<MODE>(a, g[i].count, w, s);
            whole[i] = w * ncol;
            small[i] = s * ncol;
            if (MODE == kDw && a.accumulate && g[i].count == 0) whole[i] = 0;
        }
        mine += whole[i] + small[i];
        groups += whole[i] + small[i] > 0;
    }
    const uint32_t upto = inclusive_scan(mine, lane);
    const uint32_t all = __builtin_amdgcn_readlane(upto, 63);
    groups = inclusive_scan(groups, lane);
    const bool line = all < kFewTiles * __builtin_amdgcn_readlane(groups, 63);
    const int lo = eighth(all, xcd), hi = eighth(all, xcd + 1);
    int at = static_cast<int>(upto - mine);  // of the first of these four groups in the line
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = whole[i] + small[i], x = (xcd + 4 * lane + i) & 7;
        if (line) {
            const int from = lo <= at ? 0 : lo < at + n ? lo - at : n;
            const int to = hi <= at ? 0 : hi < at + n ? hi - at : n;
            g[i].start = from < whole[i] ? from : whole[i];
            g[i].whole = (to < whole[i] ? to : whole[i]) - g[i].start;
            g[i].column = from < whole[i] ? 0 : from - whole[i];
            g[i].tiles = to - from;
        } else {
            g[i].start = eighth(whole[i], x);
            g[i].whole = eighth(whole[i], x + 1) - g[i].start;
            g[i].column = eighth(small[i], x);
            g[i].tiles = g[i].whole + eighth(small[i], x + 1) - g[i].column;
        }
        at += n;
        g[i].before = static_cast<int>(sum);
        sum += g[i].tiles;
    }
    const uint32_t incl = inclusive_scan(sum, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        g[i].before += static_cast<int>(incl - sum);
        table[4 * lane + i] = g[i];
    }
    return static_cast<int>(__builtin_amdgcn_readlane(incl, 63));
}

// The tile at `slot` of this XCD's list of `total`. If the last round of 32 (one a
// CU) has at most 16, each of them is cut into two of half the rows, for the idle
// CUs: 640 tiles of 256 x 256 x 8192 (two rounds and a half an XCD) took 523 us
// against 543 with whole tiles. `part`: which half, -1 for a whole tile.
template <int MODE>
__device__ __forceinline__ bool find(const MatmulArgs& a, const Group* table, int total, int slot, int ncol,
                                     int lane, MatTile& t, int& rt, int& ct, int& part) {
    const int over = total & (kXcdCus - 1);
    const int whole_slots = total - (over <= kXcdCus / 2 ? over : 0);
    part = -1;
    if (slot >= whole_slots) {
        part = (slot - whole_slots) & 1;
        slot = whole_slots + ((slot - whole_slots) >> 1);
        if (slot >= total) return false;
    }
    int e = -1;
    Group g{};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Group h = table[4 * lane + i];
        if (slot >= h.before && slot < h.before + h.tiles) {
            e = 4 * lane + i;
            g = h;
        }
    }
    const int src = __builtin_amdgcn_readfirstlane(
        __ffsll(static_cast<unsigned long long>(__ballot(e >= 0))) - 1);
    t.group = __builtin_amdgcn_readlane(e, src);
    slot -= __builtin_amdgcn_readlane(g.before, src);
    const int mine = __builtin_amdgcn_readlane(g.whole, src);
    int first = __builtin_amdgcn_readlane(g.first, src);
    t.nrows = __builtin_amdgcn_readlane(g.count, src);
    int whole, small;
    row_tiles<MODE>(a, t.nrows, whole, small);
    if (slot < mine) {
        // bands of equal height, at most kBand row tiles, column by column
        const uint32_t lin = slot + __builtin_amdgcn_readlane(g.start, src);
        const uint32_t bands = (static_cast<uint32_t>(whole) + kBand - 1) / kBand;
        const uint32_t height = (whole + bands - 1) / bands, span = height * ncol;
        const uint32_t band = lin / span, within = lin - band * span;
        const uint32_t left = whole - band * height, here = left < height ? left : height;
        const uint32_t col = within / here;
        rt = __builtin_amdgcn_readfirstlane(static_cast<int>(band * height + within - col * here));
        ct = __builtin_amdgcn_readfirstlane(static_cast<int>(col));
    } else {
        rt = whole;
        ct = slot - mine + __builtin_amdgcn_readlane(g.column, src);
    }
    if (MODE != kDw) {
        first += rt * BM;
        t.nrows -= rt * BM;
        t.nrows = t.nrows < BM ? t.nrows : BM;
    }
    t.row0 = first;
    return true;
}

// Half `h` of an operand: index i (0..127) in the half -> index in the tile. Of A the
// first 64 are the rows of waves 0..3 and the last those of waves 4..7, `each` rows
// apart (64, or fewer in the last half of a tile's rows).
template <bool B>
__device__ __forceinline__ int half_index(int i, int h, int each) {
    if (B) return (i >> 5) * 64 + h * 32 + (i & 31);
    return h * 128 + (i >> 6) * each + (i & 63);
}

// Rows of `rows` (1..128) that each half of the waves takes: whole sub-tiles of 16.
__device__ __forceinline__ int rows_each(int rows) { return (rows + 31) >> 5 << 4; }

// Staging of the halves of an operand: two 1 KB loads a wave and half.
template <bool TR, bool B>
struct HalfStager {
    const uint8_t* base;
    uint32_t off[2][2];

    static __device__ __forceinline__ int row(int i, int wave, int lane) {  // of the half in LDS
        return TR ? (wave + 8 * i) * 4 + (lane >> 4) : (wave + 8 * i) * 8 + (lane >> 3);
    }
    static __device__ __forceinline__ int piece(int i, int wave, int lane) {
        const int r = row(i, wave, lane);
        return TR ? (lane & 15) ^ red_spread<128>(r) : (lane & 7) ^ row_spread(r);
    }
    __device__ __forceinline__ void init(const uint16_t* p, int64_t ld, int valid, int each0, int each1,
                                         int wave, int lane) {
        base = reinterpret_cast<const uint8_t*>(uniform(reinterpret_cast<uint64_t>(p)));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = row(i, wave, lane), c = piece(i, wave, lane) * 8;
                int m = half_index<B>(TR ? c : r, h, h ? each1 : each0);
                m = m < valid ? m : valid - (TR ? 8 : 1);
                off[h][i] = static_cast<uint32_t>((TR ? r * ld + m : m * ld + c) * 2);
            }
    }
    // step k; ld: of the operand, red: length of the reduction
    __device__ __forceinline__ void load(uint32_t lds, int h, int k, int ld, int red, int wave, int lane) const {
        const uint8_t* b = base + static_cast<int64_t>(k) * (TR ? kStepR * 2 * ld : kStepR * 2);
        const int left = red - k * kStepR;
        if (left >= kStepR) {
#pragma unroll
            for (int i = 0; i < 2; ++i) lds_load16(b, off[h][i], lds + (wave + 8 * i) * 1024);
        } else {
            // opaque, so that nothing of this is computed ahead of the loop and kept
            asm volatile("" : "+v"(lane));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = TR ? row(i, wave, lane) : piece(i, wave, lane) * 8;
                const void* src = at < left ? static_cast<const void*>(b + off[h][i])
                                            : static_cast<const void*>(g_zero16);
                lds_load16(src, lds + (wave + 8 * i) * 1024);
            }
        }
    }
};

constexpr int A0 = 0, B0 = kHalf, B1 = 2 * kHalf, A1 = 3 * kHalf;  // halves of a stage

// A tile with its requests under way.
template <int MODE>
struct Work {
    static constexpr bool AT = MODE == kDw, BT = MODE != kFwd;
    HalfStager<AT, false> sa;
    HalfStager<BT, true> sb;
    int red, steps, rows, cols, col0;
    int64_t out_row;
    bool small;

    __device__ __forceinline__ void load_a(const MatmulArgs& a, uint32_t p, int h, int k, int wave, int lane) const {
        sa.load(p, h, k, static_cast<int>(MODE == kFwd ? a.K : a.N), red, wave, lane);
    }
    // phase 0's halves of step k
    __device__ __forceinline__ void request(const MatmulArgs& a, uint32_t p, int k, int wave, int lane) const {
        load_a(a, p + A0, 0, k, wave, lane);
        sb.load(p + B0, 0, k, static_cast<int>(a.K), red, wave, lane);
        sb.load(p + B1, 1, k, static_cast<int>(a.K), red, wave, lane);
    }
    // steps 0 and 1 but for step 1's A1: 6 + 2 + 6 loads a wave (small tiles: 6 + 6)
    __device__ __forceinline__ void start(const MatmulArgs& a, const Operands<MODE>& o, uint32_t at, int wave,
                                          int lane) {
        red = __builtin_amdgcn_readfirstlane(static_cast<int>(o.red));
        rows = __builtin_amdgcn_readfirstlane(o.rows);
        cols = __builtin_amdgcn_readfirstlane(o.cols);
        col0 = __builtin_amdgcn_readfirstlane(static_cast<int>(o.col0));
        out_row = uniform(o.out_row);
        small = rows <= BM / 2;
        steps = (red + kStepR - 1) / kStepR;
        if (steps == 0) return;
        sa.init(o.a, o.lda, rows, small ? rows_each(rows) : 64, small ? 0 : rows_each(rows - 128), wave, lane);
        sb.init(o.b, o.ldb, cols, 0, 0, wave, lane);
        request(a, at, 0, wave, lane);
        if (!small) load_a(a, at + A1, 1, 0, wave, lane);
        if (steps > 1) request(a, at + (small ? 3 * kHalf : 4 * kHalf), 1, wave, lane);
    }
};

}  // namespace

// The products of a tile that `start` has been called for; then `next()`, which may
// request the next tile's first steps, then the stores.
template <int MODE, bool LINEAR, bool SMALL, typename Next>
__device__ __forceinline__ void run_tile(const MatmulArgs& a, const Work<MODE>& w, uint8_t* lds, int wave,
                                         int lane, Next&& next) {
    const int wm = wave >> 2, wn = wave & 3;
    Reader<Work<MODE>::AT, 128> ra;
    Reader<Work<MODE>::BT, 128> rb;
    ra.init(wm * 64, lane);
    rb.init(wn * 32, lane);

    constexpr int MI = SMALL ? 4 : 8;
    f32x4 acc[MI][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int steps = w.steps;
    const int each = SMALL ? rows_each(w.rows) : rows_each(w.rows - 128), subs = each >> 4;
    const uint32_t at = lds_address(lds);
    constexpr int kStage = SMALL ? 3 * kHalf : 4 * kHalf;

    bf16x8 fa[4][2], fb[4][2];
    auto read_a = [&](const uint8_t* p) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i][s] = ra.read(p, i, s);
    };
    auto read_b = [&](const uint8_t* p) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[j][s] = rb.read(p + (j < 2 ? B0 : B1), j & 1, s);
    };
    auto reads_done = [&]() __attribute__((always_inline)) { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
    // the products of half ih with sub-tiles of rows: all 4, or the first `subs`
    auto multiply = [&](int ih, int subs) __attribute__((always_inline)) {
        block_barrier();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i > 0 && i >= subs) continue;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[4 * ih + i][j] = mfma_bf16(fb[j][s], fa[i][s], acc[4 * ih + i][j]);
                // in this order: the two products of one accumulator stay four apart (the
                // scheduler put them side by side in some builds, 13 % slower)
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        block_barrier();
    };
    if (steps > 0) {
        // step 0's halves of phase 0 have landed
        if (steps > 1) wait_loads<SMALL ? 6 : 8>();
        else wait_loads<SMALL ? 0 : 2>();
        block_barrier();
        if (wave >= 4) block_barrier();  // half a phase behind

        int so = 0;  // stage of step k
        for (int k = 0; k < steps; ++k) {
            const int left = steps - 1 - k;
            const uint8_t* cur = lds + so;
            read_b(cur);
            read_a(cur + A0);
            if (SMALL) {
                // step k + 2 over step k - 1's stage; step k + 1 has landed
                if (left > 1) {
                    w.request(a, at + (so == 0 ? 2 * kStage : so - kStage), k + 2, wave, lane);
                    wait_loads<6>();
                } else {
                    wait_loads<0>();
                }
                reads_done();
                multiply(0, subs);
                so = so == 2 * kStage ? 0 : so + kStage;
                continue;
            }
            // phase 0: A1 of step k + 1; A1 of this step has landed
            if (left > 0) {
                w.load_a(a, at + (kStage - so) + A1, 1, k + 1, wave, lane);
                wait_loads<8>();
            } else {
                wait_loads<0>();
            }
            reads_done();
            multiply(0, 4);
            // phase 1: A0, B0 and B1 of step k + 2; those of step k + 1 have landed
            read_a(cur + A1);
            if (left > 1) {
                w.request(a, at + so, k + 2, wave, lane);
                wait_loads<8>();
            } else if (left == 1) {
                wait_loads<2>();
            }
            reads_done();
            multiply(1, subs);
            so = kStage - so;
        }
        if (wave < 4) block_barrier();
    }
    // all waves have read all of LDS
    const int rows = w.rows, cols = w.cols, col0 = w.col0;
    const int64_t out_row = w.out_row, ldo = MODE == kFwd ? a.N : a.K;
    next();

    // opaque, so that the addresses are not computed once for all tiles and kept
    asm volatile("" : "+v"(lane));
    store_all<MODE, LINEAR, MI, 2>(
        a, acc, Place{out_row, ldo, col0, rows, wn * 64, cols},
        [&](int i) {
            if ((SMALL || i >= 4) && (i & 3) > 0 && (i & 3) >= subs) return -1000000;
            return (SMALL ? wm * each : i < 4 ? wm * 64 : 128 + wm * each) + 16 * (i & 3);
        },
        lane);
}

// Blocks walk their XCD's tiles in a round robin; a block requests its next tile's
// first two steps before it stores a tile.
template <int MODE, bool LINEAR>
__global__ __launch_bounds__(64 * kWaves, 2) void matmul256_kernel(MatmulArgs a) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t at = lds_address(lds);
    Group* table = reinterpret_cast<Group*>(lds + kStages);
    const int ncol = static_cast<int>(((MODE == kFwd ? a.N : a.K) + BN - 1) / BN);
    const int total = fill_table<MODE>(a, table, ncol, lane);
    __syncthreads();

    int slot = blockIdx.x >> 3;
    const int stride = gridDim.x >> 3;
    // the tile that the block does after the one it is at: found while that one's
    // first loads are under way, requested when its products are done
    MatTile t;
    int rt, ct, part;
    bool more;
    auto find_next = [&]() __attribute__((always_inline)) {
        int lane_ = lane;
        asm volatile("" : "+v"(lane_));  // as in run_tile: nothing kept in registers for the next tile
        do {
            more = find<MODE>(a, table, total, slot, ncol, lane_, t, rt, ct, part);
            slot += stride;
            // the second half of a cut tile may have no rows
        } while (more && part > 0 && (MODE == kDw ? a.N - rt * BM : t.nrows) <= BM / 2);
    };
    Work<MODE> w;
    auto start = [&]() __attribute__((always_inline)) {
        int lane_ = lane;
        asm volatile("" : "+v"(lane_));
        if (more) w.start(a, operands<MODE, BM, BN>(a, t, rt, ct, part), at, wave, lane_);
    };
    find_next();
    if (!more) return;
    start();
    for (bool going = true; going;) {
        const bool small = w.small;
        find_next();
        going = more;
        if (small) run_tile<MODE, LINEAR, true>(a, w, lds, wave, lane, start);
        else run_tile<MODE, LINEAR, false>(a, w, lds, wave, lane, start);
    }
}

// Blocks that have a tile, an upper bound: the host does not know the group sizes.
template <int MODE>
static int64_t matmul256_blocks(const MatmulArgs& a) {
    const int64_t ncol = ((MODE == kFwd ? a.N : a.K) + BN - 1) / BN;
    if (MODE == kDw) {
        // each group's eighth rounds up by less than a tile; cut tiles
        return 8 * (a.E * ((a.N + BM - 1) / BM * ncol / 8 + 1) + kXcdCus / 2);
    }
    // an XCD's shares of a group's two kinds round up by less than a tile each; cut tiles
    const int64_t groups = a.E < a.P ? a.E : a.P;
    return 8 * ((a.P / BM + groups) * ncol / 8 + 2 * groups + 1 + kXcdCus / 2);
}

template <int MODE, bool LINEAR>
static hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
    static LdsDevices allowed;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(&matmul256_kernel<MODE, LINEAR>),
                                   kStages + kTable, allowed);
    if (e != hipSuccess) return e;
    // Persistent blocks, one a CU, where the tiles cost about the same (a dense
    // product) or are short (weight gradients): 16 experts of 512 rows, 5120 x 8192,
    // 822 us against 886 with a block a tile. Tiles of ragged groups differ in cost,
    // which a block a tile balances: 16 experts, 8192 rows, 16384 x 5120, dx 1405
    // against 1554 us (forward 1301 against 1304).
    int64_t blocks = matmul256_blocks<MODE>(a);
    if ((MODE == kDw || a.E == 1) && blocks > 256) blocks = 256;
    if (blocks > kGridX) blocks = kGridX;  // of several tiles each
    hipLaunchKernelGGL((matmul256_kernel<MODE, LINEAR>), dim3(static_cast<unsigned>(blocks)),
                       dim3(64 * kWaves), kStages + kTable, stream, a);
    return hipGetLastError();
}

hipError_t launch_matmul256(int mode, bool linear, const MatmulArgs& a, hipStream_t stream) {
    if (mode == kDx) return launch<kDx, false>(a, stream);
    if (mode == kDw) return launch<kDw, false>(a, stream);
    return linear ? launch<kFwd, true>(a, stream) : launch<kFwd, false>(a, stream);
}

}  // namespace moe
