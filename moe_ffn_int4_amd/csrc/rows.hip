// rows.hip -- the row operators between the products: SwiGLU, the gradient through
// an activation, and expert rows moved to and from their tokens. Each reads and
// writes its operands once, in 16-byte pieces of 8 bf16 values; HBM bounds them all.
#include "common.h"
#include "train.h"

namespace moe {

namespace {

constexpr int NT = 256;

__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}
__device__ __forceinline__ void save8(uint16_t* p, const float* v) {
    *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                                         pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7])};
}

// Rows of `pieces` 16-byte pieces over blocks of 256 threads: 1 << shift threads a
// row (a power of two covering the row, at most the block), chunks of a row across
// blocks when it is longer.
struct RowGrid {
    int shift;
    unsigned chunks;
    unsigned blocks;
    bool ok;
};

RowGrid row_grid(int64_t rows, int64_t pieces) {
    RowGrid g;
    g.shift = 0;
    while ((1 << g.shift) < NT && (1 << g.shift) < pieces) ++g.shift;
    g.chunks = static_cast<unsigned>((pieces + (1 << g.shift) - 1) >> g.shift);
    const int64_t per = NT >> g.shift;
    const int64_t blocks = (rows + per - 1) / per * g.chunks;
    g.ok = blocks <= 0x7FFFFFFF;
    g.blocks = static_cast<unsigned>(blocks);
    return g;
}

// this thread's row and piece; false past the end
__device__ __forceinline__ bool row_piece(int64_t rows, int64_t pieces, int shift, unsigned chunks,
                                          int64_t& row, int64_t& piece) {
    const unsigned block = block_index(), b = block / chunks;
    row = (static_cast<int64_t>(b) << (8 - shift)) + (threadIdx.x >> shift);
    piece = (static_cast<int64_t>(block - b * chunks) << shift) + (threadIdx.x & ((1 << shift) - 1));
    return row < rows && piece < pieces;
}
static_assert(NT == 256, "row_piece: 2^8 threads");

}  // namespace

// ------------------------------------------------------------------- SwiGLU

__global__ __launch_bounds__(NT) void swiglu_kernel(const uint16_t* __restrict__ z, int64_t rows, int64_t h,
                                                    int shift, unsigned chunks, uint16_t* __restrict__ y) {
    int64_t r, c;
    if (!row_piece(rows, h / 8, shift, chunks, r, c)) return;
    float g[8], u[8];
    load8(z + r * 2 * h + c * 8, g);
    load8(z + r * 2 * h + h + c * 8, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = g[i] * sigmoid_rn(g[i]) * u[i];
    save8(y + r * h + c * 8, g);
}

// dz may be z: a thread reads the two pieces that it then writes
__global__ __launch_bounds__(NT) void swiglu_backward_kernel(const uint16_t* __restrict__ dy, const uint16_t* z,
                                                             int64_t rows, int64_t h, int shift,
                                                             unsigned chunks, uint16_t* dz) {
    int64_t r, c;
    if (!row_piece(rows, h / 8, shift, chunks, r, c)) return;
    float d[8], g[8], u[8];
    load8(dy + r * h + c * 8, d);
    load8(z + r * 2 * h + c * 8, g);
    load8(z + r * 2 * h + h + c * 8, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s = sigmoid_rn(g[i]);
        // the bound as in act_slope
        const float c = __builtin_amdgcn_fmed3f(g[i], -90.0f, 90.0f);
        u[i] = d[i] * u[i] * fmaf(c * s, 1.0f - s, s);
        g[i] = d[i] * (g[i] * s);
    }
    save8(dz + r * 2 * h + c * 8, u);
    save8(dz + r * 2 * h + h + c * 8, g);
}

hipError_t launch_swiglu(const uint16_t* z, int64_t rows, int64_t h, uint16_t* y, hipStream_t stream) {
    const RowGrid g = row_grid(rows, h / 8);
    if (!g.ok) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(swiglu_kernel, block_grid(g.blocks), dim3(NT), 0, stream, z, rows, h, g.shift, g.chunks, y);
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const uint16_t* dy, const uint16_t* z, int64_t rows, int64_t h,
                                  uint16_t* dz, hipStream_t stream) {
    const RowGrid g = row_grid(rows, h / 8);
    if (!g.ok) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(swiglu_backward_kernel, block_grid(g.blocks), dim3(NT), 0, stream, dy, z, rows, h, g.shift,
                       g.chunks, dz);
    return hipGetLastError();
}

// ------------------------------------------------------ gradient of an activation

// A block takes `rows` rows from blockIdx.y * rows and up to 64 pieces of columns;
// lanes (a power of two covering the columns, at most 64) walk the columns and the
// block's other threads the rows, two at a time. Each thread sums its rows, the
// block its threads in order, and dz_finish the slices in order. ACT is a template
// argument: the switch would be taken for every value.
template <int ACT>
__global__ __launch_bounds__(NT) void linear_dz_kernel(const uint16_t* dy, const uint16_t* z, int64_t T,
                                                       int64_t N, int shift, int64_t rows, uint16_t* dz,
                                                       float* __restrict__ sums) {
    __shared__ float part[NT * 8];
    const int64_t c = (static_cast<int64_t>(blockIdx.x) << shift) + (threadIdx.x & ((1 << shift) - 1));
    const int first = threadIdx.x >> shift, stride = NT >> shift;
    const int64_t r0 = blockIdx.y * rows, r1 = r0 + rows < T ? r0 + rows : T;
    float sum[8] = {};
    auto one = [&](float* d, const float* v, int64_t at) __attribute__((always_inline)) {
        if (ACT != MOE_ACT_NONE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= act_slope(v[i], ACT);
            save8(dz + at, d);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += d[i];
    };
    if (c * 8 < N) {
        const int64_t step = stride * N;
        int64_t at = (r0 + first) * N + c * 8, r = r0 + first;
        for (; r + stride < r1; r += 2 * stride, at += 2 * step) {
            float d0[8], d1[8], v0[8], v1[8];
            load8(dy + at, d0);
            load8(dy + at + step, d1);
            if (ACT != MOE_ACT_NONE) {
                load8(z + at, v0);
                load8(z + at + step, v1);
            }
            one(d0, v0, at);
            one(d1, v1, at + step);
        }
        if (r < r1) {
            float d0[8], v0[8];
            load8(dy + at, d0);
            if (ACT != MOE_ACT_NONE) load8(z + at, v0);
            one(d0, v0, at);
        }
    }
    if (!sums) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.x * 8 + i] = sum[i];
    __syncthreads();
    // thread -> one column of the block's 8 << shift; a loop because there may be
    // more columns than threads
    for (int col = threadIdx.x; col < (8 << shift); col += NT) {
        const int64_t at = (static_cast<int64_t>(blockIdx.x) << (shift + 3)) + col;
        if (at >= N) break;
        float s = 0.f;
        for (int i = 0; i < stride; ++i) s += part[(i << (shift + 3)) + col];
        sums[blockIdx.y * N + at] = s;
    }
}

// Up to 512 rows: all of 64 columns in one block of 16 waves, eight lanes a row, four rows a
// thread, all loaded at once; the rows of a wave are added across lanes, the waves in order. One
// launch: 126 x 2968 takes 4.1 us instead of 5.8 in a graph, 9.7 instead of 12 called one by
// one; 508 x 2104 8.0 (7.7) and 10.0 (12.4). At 1024 rows the arithmetic of so few blocks
// shows: 13.1 against 4.9 for 64 columns.
constexpr int kDzWaves = 16;
constexpr int kDzUnder = 4;
constexpr int64_t kDzOneLaunch = kDzWaves * 8 * kDzUnder;
template <int ACT>
__global__ __launch_bounds__(64 * kDzWaves) void linear_dz_columns_kernel(const uint16_t* dy, const uint16_t* z,
                                                                          int64_t T, int64_t N, uint16_t* dz,
                                                                          float* __restrict__ db) {
    __shared__ float part[kDzWaves * 64];
    constexpr int kRows = kDzWaves * 8;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x & 7);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r0 = threadIdx.x >> 3;
    float sum[8] = {};
    if (c * 8 < N && r0 < T) {
        float d[kDzUnder][8], v[kDzUnder][8];
#pragma unroll
        for (int u = 0; u < kDzUnder; ++u) {
            // rows past the end load the last one, for nothing: a branch would wait for each load
            const int64_t r = r0 + u * kRows < T ? r0 + u * kRows : T - 1;
            load8(dy + r * N + c * 8, d[u]);
            if (ACT != MOE_ACT_NONE) load8(z + r * N + c * 8, v[u]);
        }
#pragma unroll
        for (int u = 0; u < kDzUnder; ++u) {
            const int64_t r = r0 + u * kRows;
            if (r >= T) break;
            if (ACT != MOE_ACT_NONE) {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[u][i] *= act_slope(v[u][i], ACT);
                save8(dz + r * N + c * 8, d[u]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += d[u][i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int off = 8; off < 64; off <<= 1) sum[i] += __shfl_xor(sum[i], off, kWave);
    }
    if (lane < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) part[wave * 64 + lane * 8 + i] = sum[i];
    }
    __syncthreads();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (threadIdx.x >= 64 || col >= N || !db) return;
    float s = part[threadIdx.x];
#pragma unroll
    for (int w = 1; w < kDzWaves; ++w) s += part[w * 64 + threadIdx.x];
    db[col] = s;
}

// A block adds the slices of 32 columns: eight threads a column take every eighth slice,
// and their sums are added in order. (One thread a column: 128 loads in a row.)
__global__ __launch_bounds__(NT) void dz_finish_kernel(const float* __restrict__ partial, int slices, int64_t N,
                                                       float* __restrict__ db) {
    __shared__ float part[NT];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
    float s = 0.f;
    if (c < N) {
#pragma unroll 8
        for (int i = threadIdx.x >> 5; i < slices; i += 8) s += partial[i * N + c];
    }
    part[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x >= 32 || c >= N) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) s += part[i * 32 + threadIdx.x];
    db[c] = s;
}

constexpr int64_t kDzRows = 64;
constexpr int64_t kDzBlocks = 512;
constexpr int64_t kDzMaxSlices = 1024;

// log2 of the lanes that cover a row's pieces, at most 64
static int dz_shift(int64_t N) {
    int shift = 0;
    while ((1 << shift) < 64 && (8 << shift) < N) ++shift;
    return shift;
}

// Slices of the rows: 64 rows each, shorter ones while there are fewer than kDzBlocks
// blocks and each thread has a row (gelu, us: 800 x 3032 9.1 against 12.9 in slices of 64,
// 3655 x 944 10.3 against 15.1; with 128, 256 and 1024 blocks 10.5, 9.5, 10.2 and 12.7, 10.0,
// 11.7). One for what linear_dz_columns_kernel takes.
int64_t linear_dz_slices(int64_t T, int64_t N) {
    const int shift = dz_shift(N);
    const int64_t cols = (N + (8 << shift) - 1) >> (shift + 3), stride = NT >> shift;
    if (T <= kDzOneLaunch) return 1;
    int64_t s = (kDzBlocks + cols - 1) / cols;
    const int64_t most = (T + stride - 1) / stride, least = (T + kDzRows - 1) / kDzRows;
    s = s < most ? s : most;
    s = s < least ? least : s;
    return s < kDzMaxSlices ? s : kDzMaxSlices;
}

hipError_t launch_linear_dz(const uint16_t* dy, const uint16_t* z, int act, int64_t T, int64_t N,
                            uint16_t* dz, float* db, float* partial, hipStream_t stream) {
    const int64_t slices = linear_dz_slices(T, N);
    if (slices == 1) {
        auto* one = act == MOE_ACT_RELU        ? linear_dz_columns_kernel<MOE_ACT_RELU>
                    : act == MOE_ACT_SILU      ? linear_dz_columns_kernel<MOE_ACT_SILU>
                    : act == MOE_ACT_GELU      ? linear_dz_columns_kernel<MOE_ACT_GELU>
                    : act == MOE_ACT_GELU_TANH ? linear_dz_columns_kernel<MOE_ACT_GELU_TANH>
                                               : linear_dz_columns_kernel<MOE_ACT_NONE>;
        hipLaunchKernelGGL(one, dim3(static_cast<unsigned>((N + 63) / 64)), dim3(64 * kDzWaves), 0, stream, dy, z, T,
                           N, dz, db);
        return hipGetLastError();
    }
    const int64_t rows = (T + slices - 1) / slices;
    const int shift = dz_shift(N);
    const int64_t cols = (N + (8 << shift) - 1) >> (shift + 3);
    float* sums = db ? partial : nullptr;
    auto* kernel = act == MOE_ACT_RELU        ? linear_dz_kernel<MOE_ACT_RELU>
                   : act == MOE_ACT_SILU      ? linear_dz_kernel<MOE_ACT_SILU>
                   : act == MOE_ACT_GELU      ? linear_dz_kernel<MOE_ACT_GELU>
                   : act == MOE_ACT_GELU_TANH ? linear_dz_kernel<MOE_ACT_GELU_TANH>
                                              : linear_dz_kernel<MOE_ACT_NONE>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(cols), static_cast<unsigned>(slices)), dim3(NT), 0,
                       stream, dy, z, T, N, shift, rows, dz, sums);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !db) return e;
    hipLaunchKernelGGL(dz_finish_kernel, dim3(static_cast<unsigned>((N + 31) / 32)), dim3(NT), 0, stream,
                       partial, static_cast<int>(slices), N, db);
    return hipGetLastError();
}

// ------------------------------------------------------------ expert row movement

__global__ __launch_bounds__(NT) void permute_rows_kernel(const uint16_t* __restrict__ x,
                                                          const int32_t* __restrict__ perm, int64_t T,
                                                          int top_k, int64_t d, int shift, unsigned chunks,
                                                          uint16_t* __restrict__ xp) {
    int64_t s, c;
    if (!row_piece(T * top_k, d / 8, shift, chunks, s, c)) return;
    const int pair = perm[s];
    u32x4 v = {0, 0, 0, 0};  // a pair outside [0, T * top_k) gives a row of zeros
    if (pair >= 0 && pair < T * top_k)
        v = *reinterpret_cast<const u32x4*>(x + static_cast<int64_t>(pair / top_k) * d + c * 8);
    *reinterpret_cast<u32x4*>(xp + s * d + c * 8) = v;
}

template <typename O>
__global__ __launch_bounds__(NT) void combine_rows_kernel(const O* __restrict__ o,
                                                          const int32_t* __restrict__ inv,
                                                          const float* __restrict__ gates,
                                                          const uint16_t* residual, int64_t T, int top_k,
                                                          int64_t d, int shift, unsigned chunks, uint16_t* y) {
    int64_t t, c;
    if (!row_piece(T, d / 8, shift, chunks, t, c)) return;
    float acc[8] = {};
    if (residual) load8(residual + t * d + c * 8, acc);
    // four rows under way at once: the indices, then the rows, then the sums in order
    // (8192 x 8 x 5120: 166 us, one at a time 172)
    for (int j0 = 0; j0 < top_k; j0 += 4) {
        int slot[4];
        float g[4], v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u;
            slot[u] = j < top_k ? inv[t * top_k + j] : -1;
            g[u] = j < top_k && gates ? gates[t * top_k + j] : 1.0f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (slot[u] >= 0 && slot[u] < T * top_k) load8(o + static_cast<int64_t>(slot[u]) * d + c * 8, v[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (slot[u] >= 0 && slot[u] < T * top_k) {
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(g[u], v[u][i], acc[i]);
            }
    }
    save8(y + t * d + c * 8, acc);
}

// d_o[slot] = g dy[t] and d_gates[t, j] = <dy[t], o[slot]>: a wave for each (token, j), or,
// for rows of up to 256 values, 1 << shift lanes that cover the row. (6221 x 8 x 80: 8.4 against 18.9
// us with whole waves, 16384 x 8 x 256 36 against 50. As one kernel with runtime lanes,
// 8192 x 8 x 520 took 42 instead of 34.)
template <typename O, bool WAVE>
__global__ __launch_bounds__(NT) void combine_backward_kernel(const uint16_t* __restrict__ dy,
                                                              const O* __restrict__ o,
                                                              const int32_t* __restrict__ inv,
                                                              const float* __restrict__ gates, int64_t T,
                                                              int top_k, int64_t d, int shift_,
                                                              uint16_t* __restrict__ d_o,
                                                              float* __restrict__ d_gates) {
    const int shift = WAVE ? 6 : shift_, lanes = 1 << shift, lane = threadIdx.x & (lanes - 1);
    const int64_t pair = (static_cast<int64_t>(block_index()) << (8 - shift)) + (threadIdx.x >> shift);
    if (pair >= T * top_k) return;
    const int64_t t = pair / top_k;
    const int slot = inv[pair];
    const bool in = slot >= 0 && slot < T * top_k;
    const float g = gates ? gates[pair] : 1.0f;
    float dot = 0.f;
    const uint16_t* from = dy + t * d;
    const int64_t row = static_cast<int64_t>(slot) * d, pieces = in ? d / 8 : 0;
    // four pieces of each operand under way at once
    for (int64_t c0 = lane; c0 < pieces; c0 += 4 * lanes) {
        float v[4][8], w[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t c = c0 + u * lanes;
            if (c >= pieces) continue;
            load8(from + c * 8, v[u]);
            if (d_gates) load8(o + row + c * 8, w[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t c = c0 + u * lanes;
            if (c >= pieces) continue;
            if (d_gates) {
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = fmaf(v[u][i], w[u][i], dot);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] *= g;
            save8(d_o + row + c * 8, v[u]);
        }
    }
    if (!d_gates) return;
    if (WAVE) dot = wave_sum(dot);
    else
        for (int off = lanes >> 1; off > 0; off >>= 1) dot += __shfl_xor(dot, off, kWave);
    if (lane == 0) d_gates[pair] = dot;
}

hipError_t launch_permute_rows(const uint16_t* x, const int32_t* perm, int64_t T, int top_k, int64_t d,
                               uint16_t* xp, hipStream_t stream) {
    const RowGrid g = row_grid(T * top_k, d / 8);
    if (!g.ok) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(permute_rows_kernel, block_grid(g.blocks), dim3(NT), 0, stream, x, perm, T, top_k, d, g.shift,
                       g.chunks, xp);
    return hipGetLastError();
}

hipError_t launch_combine_rows(const void* o, bool o_fp32, const int32_t* inv, const float* gates,
                               const uint16_t* residual, int64_t T, int top_k, int64_t d, uint16_t* y,
                               hipStream_t stream) {
    const RowGrid g = row_grid(T, d / 8);
    if (!g.ok) return hipErrorInvalidConfiguration;
    if (o_fp32)
        hipLaunchKernelGGL(combine_rows_kernel<float>, block_grid(g.blocks), dim3(NT), 0, stream,
                           static_cast<const float*>(o), inv, gates, residual, T, top_k, d, g.shift, g.chunks, y);
    else
        hipLaunchKernelGGL(combine_rows_kernel<uint16_t>, block_grid(g.blocks), dim3(NT), 0, stream,
                           static_cast<const uint16_t*>(o), inv, gates, residual, T, top_k, d, g.shift, g.chunks, y);
    return hipGetLastError();
}

hipError_t launch_combine_backward(const uint16_t* dy, const void* o, bool o_fp32, const int32_t* inv,
                                   const float* gates, int64_t T, int top_k, int64_t d, uint16_t* d_o,
                                   float* d_gates, hipStream_t stream) {
    int shift = 0;
    while ((1 << shift) < 64 && (8 << shift) < d) ++shift;
    const int64_t per = NT >> shift, blocks = (T * top_k + per - 1) / per;
    const dim3 grid = block_grid(blocks);
    auto launch = [&](auto* kernel, auto* rows) {
        hipLaunchKernelGGL(kernel, grid, dim3(NT), 0, stream, dy, rows, inv, gates, T, top_k, d, shift, d_o, d_gates);
    };
    const auto* o32 = static_cast<const float*>(o);
    const auto* o16 = static_cast<const uint16_t*>(o);
    if (o_fp32)
        shift == 6 ? launch(&combine_backward_kernel<float, true>, o32) : launch(&combine_backward_kernel<float, false>, o32);
    else
        shift == 6 ? launch(&combine_backward_kernel<uint16_t, true>, o16)
                   : launch(&combine_backward_kernel<uint16_t, false>, o16);
    return hipGetLastError();
}

}  // namespace moe
