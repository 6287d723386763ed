// train.h -- launchers of the operators beside the layer's forward: grouped and
// dense products with their gradients, SwiGLU, expert row movement (internal to
// the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "moe_int4.h"

namespace moe {

// products of matmul.h
constexpr int kFwd = 0;
constexpr int kDx = 1;
constexpr int kDw = 2;

struct MatmulArgs {
    const uint16_t* a;       // kFwd: x [P, K]; kDx, kDw: dy [P, N]
    const uint16_t* b;       // kFwd, kDx: W [E, N, K]; kDw: x [P, K]
    const int32_t* offsets;  // [E + 1] row ranges of the groups; null: one group of P rows
    int64_t P;
    int E;
    int64_t N, K;
    void* out;               // bf16, or fp32 with out_fp32
    int out_fp32;
    int accumulate;          // add to the values already in out
    // kFwd of linear: out = act(x W^T + bias) + residual, z = x W^T + bias
    const float* bias;       // [N] or null
    const uint16_t* residual;  // [P, N] or null
    uint16_t* z;             // [P, N] or null
    int act;                 // MOE_ACT_*
};

hipError_t launch_matmul256(int mode, bool linear, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_matmul_stream(bool linear, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_matmul(int mode, bool linear, const MatmulArgs& a, hipStream_t stream);

// two fp32 -> packed bf16 pair, round to nearest even, NaN kept
__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}

// Activations and their derivatives, in fp32. For z < -88 exp(-z) overflows to
// infinity and the sigmoid is 0, its limit, so no range check is needed there.
__device__ __forceinline__ float sigmoid_rn(float z) { return 1.0f / (1.0f + __expf(-z)); }

__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case MOE_ACT_RELU: return z < 0.0f ? 0.0f : z;  // keeps NaN
        case MOE_ACT_SILU: return z * sigmoid_rn(z);
        case MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        case MOE_ACT_GELU_TANH: {
            // 0.5 (1 + tanh(u)) = sigmoid(2 u)
            const float u = 1.5957691216057308f * fmaf(0.044715f * z * z, z, z);
            return z * sigmoid_rn(u);
        }
        default: return z;
    }
}

__device__ __forceinline__ float act_slope(float z, int act) {
    // past +-90 every slope has its limit's fp32 value; the bound keeps z^2 finite
    // (0 * infinity below) and lets NaN through
    z = z > 90.0f ? 90.0f : z < -90.0f ? -90.0f : z;
    switch (act) {
        case MOE_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
        case MOE_ACT_SILU: {
            const float s = sigmoid_rn(z);
            return fmaf(z * s, 1.0f - s, s);
        }
        case MOE_ACT_GELU:
            return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z),
                        0.5f * (1.0f + erff(z * 0.70710678118654752f)));
        case MOE_ACT_GELU_TANH: {
            const float z2 = z * z;
            const float s = sigmoid_rn(1.5957691216057308f * fmaf(0.044715f * z2, z, z));
            return fmaf(z * s * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f, z2, 1.0f), s);
        }
        default: return 1.0f;
    }
}

// dz = dy * act'(z) (bf16) and db = column sums of the unrounded dz (fp32); act
// none: db alone. Rows are summed in slices of a fixed size into `partial`
// [linear_dz_slices(T), N] and the slices in order: no atomics.
int64_t linear_dz_slices(int64_t T, int64_t N);
hipError_t launch_linear_dz(const uint16_t* dy, const uint16_t* z, int act, int64_t T, int64_t N,
                            uint16_t* dz, float* db, float* partial, hipStream_t stream);

// y = silu(g) * u of z = [g | u], rows x 2h; and its gradient
hipError_t launch_swiglu(const uint16_t* z, int64_t rows, int64_t h, uint16_t* y, hipStream_t stream);
hipError_t launch_swiglu_backward(const uint16_t* dy, const uint16_t* z, int64_t rows, int64_t h,
                                  uint16_t* dz, hipStream_t stream);

// xp[s] = x[perm[s] / top_k]; y[t] = sum_j gate[t, j] o[inv[t, j]] + residual[t], and its gradient
hipError_t launch_permute_rows(const uint16_t* x, const int32_t* perm, int64_t T, int top_k, int64_t d,
                               uint16_t* xp, hipStream_t stream);
hipError_t launch_combine_rows(const void* o, bool o_fp32, const int32_t* inv, const float* gates,
                               const uint16_t* residual, int64_t T, int top_k, int64_t d, uint16_t* y,
                               hipStream_t stream);
hipError_t launch_combine_backward(const uint16_t* dy, const void* o, bool o_fp32, const int32_t* inv,
                                   const float* gates, int64_t T, int top_k, int64_t d, uint16_t* d_o,
                                   float* d_gates, hipStream_t stream);

}  // namespace moe
