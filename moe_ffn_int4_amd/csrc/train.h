// train.h -- launchers of the operators beside the layer's forward: grouped and
// dense products with their gradients, SwiGLU, expert row movement (internal to
// the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "lds_limit.h"
#include "matmul_rule.h"
#include "moe_int4.h"

namespace moe {

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
hipError_t launch_matmul_split(int mode, bool linear, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_matmul_stream(bool linear, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_matmul(int mode, bool linear, const MatmulArgs& a, hipStream_t stream);

// A launch has fewer than 2^32 threads along x: more blocks than kGridX stand in rows of
// that many, the last of which may have blocks past the end.
constexpr int64_t kGridX = 1 << 22;
inline dim3 block_grid(int64_t blocks) {
    if (blocks <= kGridX) return dim3(static_cast<unsigned>(blocks));
    return dim3(static_cast<unsigned>(kGridX), static_cast<unsigned>((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ unsigned block_index() { return blockIdx.x + blockIdx.y * gridDim.x; }

// two fp32 -> packed bf16 pair, round to nearest even, NaN kept
__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}

// Activations and their derivatives, in fp32.

// 1 / (1 + exp(-z)): the reciprocal is good to one unit in the last place. For z <
// -88 exp(-z) overflows to infinity and the sigmoid is 0, its limit.
__device__ __forceinline__ float sigmoid_rn(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// The normal distribution's Phi(z), and e = exp(-z^2 / 2). Phi(-a) = e f(a) with f(a) =
// erfcx(a / sqrt 2) / 2, which is fitted as a polynomial of degree 8 in 1 / (1 + 0.32 a)
// to a relative 9.4e-7 over a >= 0, evaluated in fp32, so the far left tail
// keeps its relative accuracy, and the derivative shares the exponential. With the
// library's erf beside it, gelu's gradient at 8192 x 8192 took 124 us, 85 now.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float a = __builtin_fabsf(z);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.32f, a, 1.0f));
    e = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
    float p = 0.034527737647295f;  // the sum of all is 0.5: Phi(0) is exact
    p = fmaf(p, t, -0.12245695292949677f);
    p = fmaf(p, t, 0.10615243762731552f);
    p = fmaf(p, t, 0.015561919659376144f);
    p = fmaf(p, t, 0.09738484025001526f);
    p = fmaf(p, t, 0.11343652755022049f);
    p = fmaf(p, t, 0.12773366272449493f);
    p = fmaf(p, t, 0.1276598870754242f);
    p = p * t * e;
    return z < 0.0f ? p : 1.0f - p;
}

__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case MOE_ACT_RELU: return z < 0.0f ? 0.0f : z;  // keeps NaN
        case MOE_ACT_SILU: return z * sigmoid_rn(z);
        case MOE_ACT_GELU: {
            float e;
            return z * normal_cdf(z, e);
        }
        case MOE_ACT_GELU_TANH:
            // 0.5 (1 + tanh(u)) = sigmoid(2 u)
            return z * sigmoid_rn(1.5957691216057308f * fmaf(0.044715f * z * z, z, z));
        default: return z;
    }
}

__device__ __forceinline__ float act_slope(float z, int act) {
    // past +-90 every slope has its limit's fp32 value; the bounded factor keeps infinity
    // * 0 out of the products, and a NaN is still in the other factor
    const float c = __builtin_amdgcn_fmed3f(z, -90.0f, 90.0f);
    switch (act) {
        case MOE_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
        case MOE_ACT_SILU: {
            const float s = sigmoid_rn(z);
            return fmaf(c * s, 1.0f - s, s);
        }
        case MOE_ACT_GELU: {
            float e;
            const float phi = normal_cdf(z, e);
            return fmaf(c * 0.39894228040143268f, e, phi);
        }
        case MOE_ACT_GELU_TANH: {
            const float s = sigmoid_rn(1.5957691216057308f * fmaf(0.044715f * z * z, z, z));
            return fmaf(c * s * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f, c * c, 1.0f), s);
        }
        default: return 1.0f;
    }
}

// dz = dy * act'(z) (bf16) and db = column sums of the unrounded dz (fp32); act
// none: db alone. Rows are summed in slices, whose number is the sizes' alone, into `partial`
// [linear_dz_slices(T, N), N] and the slices in order: no atomics.
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
