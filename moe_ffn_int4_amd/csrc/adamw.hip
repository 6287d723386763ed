// adamw.hip -- one AdamW step over many tensors:
//   g = grad * grad_scale
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// with p the 32-bit copy where there is one, else the parameter itself.
//
// Every element is read and written once: HBM bounds it, at 28 bytes an element for bf16
// parameters and gradients with 32-bit copies and moments, at 18 with moments in 8 bits (16 as codes alone).
// A block of 256 threads takes 2048 elements of one tensor, eight a thread, all its loads
// (up to 128 bytes a thread, 112 with bf16 gradients) under way at once; a CU's eight blocks then have over 200 KB in flight. Loads
// are ordinary and stores non-temporal: 117 M bf16 parameters with copies 611 us (5.4 TB/s; a 2 GiB copy runs at 5.05), 118 M with
// fp32 gradients and moments in 8 bits 427 (5.5), as codes alone 378 (5.6). On another box, 120 M, bf16 gradients, codes alone: 620 and 339;
// with non-temporal loads 645 and 344, with ordinary stores too 623 and 349; blocks of 1024 threads 624 and 343.
//
// Moments in 8 bits: m and sqrt(v) as E4M3 codes, 128 elements sharing a scale, most / 448 of
// the block's largest magnitude (at least 2^-100). The root, not v: it halves the range of
// exponents that a code has to cover (E4M3's 2^18 of the root are 2^36 of v), and the step
// divides by it. The codes are rounded to nearest even; the update itself takes the moments
// before that rounding. The 16 threads of a block of 128 find its maximum by DPP.
//
// A code's step is 6 to 12 % of it, and a step of the moments with beta changes them by 1 - beta of what they lack, so
// codes alone stand still: sqrt(v) with beta2 = 0.999 stays 6 to 14 times too large where gradients fall to a tenth, 0.4 of its
// value where they rise fourfold, and m with beta1 = 0.99 does not follow a change of sign. What rounding to a code leaves
// is therefore kept beside it, in fourteenths of the code's step (-7 .. 7: the half step at both ends is one of the
// values), four bits a moment, a byte an element for both. These are rounded up or down with the
// probability of either's nearness, by a hash, so that their mean follows changes of any size: sqrt(v) over its value in 32
// bits is 1.000 +- 0.016 (beta2 = 0.99) or 1.000 +- 0.036 (0.999) at rest, twice that while it falls to a tenth. Codes alone are taken
// up to beta1 = 0.9 and beta2 = 0.95, where noise still carries them from code to code.
//
// Products and sums are rounded one by one, without fused multiply-adds: next to the border
// between two codes the last bit of a moment decides which it becomes, and so the codes are
// those of the formula in plain fp32 arithmetic, wherever that runs.
#include "adamw.h"

#include <math.h>

#include "common.h"
#include "train.h"

namespace moe {

namespace {

constexpr int NT = 256;
constexpr int kEach = kAdamwChunk / NT;
static_assert(kEach == 8 && kAdamwBlock == 16 * kEach, "a block of 128 is a row of 16 lanes");

enum : uint32_t {
    kParam32 = 1,  // the parameter is fp32, not bf16
    kGrad32 = 2,
    kWide = 4,     // parameter and gradient are 16-byte aligned
};

struct Tensor {
    void* param;
    const void* grad;
    float* master;
    void *m, *v;
    float *m_scale, *v_scale;
    int64_t n;
    uint32_t flags;
};

struct Factors {
    float beta1, rest1, beta2, rest2;  // rest = 1 - beta
    float keep;                        // 1 - lr wd
    float rate;                        // lr / (1 - b1^t)
    float root;                        // 1 / sqrt(1 - b2^t)
    float eps;
};

struct Args {
    Tensor t[kAdamwTensors];
    uint32_t first[kAdamwTensors];  // block of threads that starts each tensor
    uint32_t count;
    Factors f;
    // read by the kernel where they are given: then lr, step and the factors that follow from them are not the host's
    const float* grad_scale;
    const float* lr;
    const int32_t* step;
    double lr_host, log1, log2, decay;  // log of the betas
    int64_t step_host;
    int64_t fine;  // bytes from v's codes to what is kept beside both moments', or 0 for codes alone
};
static_assert(sizeof(Args) <= 4096, "a launch's arguments");

// 1 - beta^t, also where beta^t is near 1
__host__ __device__ inline double bias_fix(double log_beta, double t) { return -expm1(t * log_beta); }

__host__ __device__ inline void set_rates(Factors& f, double lr, double decay, double fix1, double fix2) {
    f.keep = static_cast<float>(1.0 - lr * decay);
    f.rate = static_cast<float>(lr / fix1);
    f.root = static_cast<float>(1.0 / sqrt(fix2));
}

template <typename T>
__device__ __forceinline__ float widen(T v) {
    if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
    else return v;
}

// eight values from p, the first `left` of them in the tensor; `wide`: in 16-byte loads
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool wide, int left, float (&x)[8]) {
    if (wide && left >= 8) {
        if constexpr (sizeof(T) == 2) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4*>(p);
            const f32x4 b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = a[i];
                x[4 + i] = b[i];
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < left ? widen(p[i]) : 0.0f;
}

template <typename T>
__device__ __forceinline__ void save8(T* p, bool wide, int left, const float (&x)[8]) {
    if (wide && left >= 8) {
        if constexpr (sizeof(T) == 2) {
            const u32x4 w = {pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]), pack_bf16x2_rn(x[4], x[5]),
                             pack_bf16x2_rn(x[6], x[7])};
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
        } else {
            const f32x4 lo = {x[0], x[1], x[2], x[3]}, hi = {x[4], x[5], x[6], x[7]};
            __builtin_nontemporal_store(lo, reinterpret_cast<f32x4*>(p));
            __builtin_nontemporal_store(hi, reinterpret_cast<f32x4*>(p) + 1);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) {
            if constexpr (sizeof(T) == 2) p[i] = static_cast<uint16_t>(pack_bf16x2_rn(x[i], 0.0f));
            else p[i] = x[i];
        }
}

// the largest of a row of 16 lanes, in all of them; NaN is passed over
__device__ __forceinline__ float row_max(float v) {
    auto step = [&v](auto ctrl) {
        const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true);
        v = fmaxf(v, __int_as_float(o));
    };
    step(std::integral_constant<int, 0xB1>{});   // lanes l ^ 1
    step(std::integral_constant<int, 0x4E>{});   // l ^ 2
    step(std::integral_constant<int, 0x141>{});  // 7 - l of each eight
    step(std::integral_constant<int, 0x140>{});  // 15 - l
    return v;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void values8(u32x2 w, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
        x[4 * i] = a[0];
        x[4 * i + 1] = a[1];
        x[4 * i + 2] = b[0];
        x[4 * i + 3] = b[1];
    }
}

// 2^e of a code's value, its step times eight; subnormals have that of 2^-6
__device__ __forceinline__ uint32_t code_power(float value) {
    const uint32_t power = __float_as_uint(value) & 0x7F800000u;
    return power > 0x3C800000u ? power : 0x3C800000u;
}

// eight codes, what is kept beside them (FINE: four bits of each byte from AT) and their block's scale
template <bool FINE, int AT>
__device__ __forceinline__ void decode8(u32x2 w, u32x2 fine, float scale, float (&x)[8]) {
#pragma clang fp contract(off)
    values8(w, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (FINE) {
            const float n = static_cast<float>(static_cast<int32_t>(fine[i / 4] << (28 - 8 * (i % 4) - AT)) >> 28);
            x[i] = x[i] + n * (__uint_as_float(code_power(x[i])) * (1.0f / 112.0f));
        }
        x[i] = x[i] * scale;
    }
}

// Two 16-bit numbers for the roundings of element e's moments. The step's number is in `seed`; m's bits give others where that
// stands still, as in a captured step that does not count.
__device__ __forceinline__ uint32_t dither(uint32_t e, uint32_t seed, float m) {
    uint32_t x = (e * 0x9E3779B1u + seed) ^ __float_as_uint(m);
    x = (x ^ x >> 15) * 0xD1B54A33u;
    x = (x ^ x >> 13) * 0x8CB92BA7u;
    return x ^ x >> 16;
}

// The codes of a block of 128 (eight values a lane of a row), and with FINE what they leave, in the four bits of each byte of `fine`
// that start at AT (zeros before), rounded by 16 bits of `random`; returns the scale.
template <bool FINE, int AT>
__device__ __forceinline__ float encode8(const float (&x)[8], const uint32_t (&random)[8], u32x2& w, u32x2& fine) {
#pragma clang fp contract(off)
    float most = 0x1p-100f;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, __builtin_fabsf(x[i]));
    most = row_max(most);
    const float inv = 448.0f * (1.0f / most);
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = x[i] * inv;
        // a NaN stays one; the largest magnitude times inv may be an ulp past 448
        c[i] = c[i] != c[i] ? c[i] : __builtin_amdgcn_fmed3f(c[i], -448.0f, 448.0f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int k = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], 0, false);
        w[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], k, true));
    }
    if (!FINE) return most / 448.0f;
    float value[8];
    values8(w, value);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // 14 / step = 112 / power; 1 / power by its exponent
        const float steps = (c[i] - value[i]) * (__uint_as_float(0x7F000000u - code_power(value[i])) * 112.0f);
        const float up = static_cast<float>(random[i] >> (AT ? 16 : 0) & 0xFFFFu) * 0x1p-16f;
        const int n = c[i] != c[i] ? 0 : static_cast<int>(floorf(steps + up));
        fine[i / 4] |= static_cast<uint32_t>(n & 15) << (8 * (i % 4) + AT);
    }
    return most / 448.0f;
}

}  // namespace

// BITS of a moment: 32; 12, a code and what it leaves; 8, a code alone
template <int BITS, bool DEVICE>
__global__ __launch_bounds__(NT) void adamw_kernel(Args a) {
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63;
    // the tensor of this block: the last that starts at or before it (each lane looks at one)
    const uint32_t start = lane < static_cast<int>(a.count) ? a.first[lane < kAdamwTensors ? lane : 0] : 0xFFFFFFFFu;
    const int at = __builtin_amdgcn_readfirstlane(__popcll(__ballot(start <= blockIdx.x)) - 1);
    const Tensor& t = a.t[at];
    const int64_t base = static_cast<int64_t>(blockIdx.x - a.first[at]) * kAdamwChunk;

    __shared__ Factors shared;
    if (DEVICE && threadIdx.x == 0) {
        Factors f = a.f;
        const double lr = a.lr ? static_cast<double>(*a.lr) : a.lr_host;
        const double s = a.step ? static_cast<double>(*a.step) : static_cast<double>(a.step_host);
        set_rates(f, lr, a.decay, bias_fix(a.log1, s), bias_fix(a.log2, s));
        shared = f;
    }

    const int64_t e = base + threadIdx.x * kEach;
    const int64_t over = t.n - e;
    const int left = over >= 8 ? 8 : over > 0 ? static_cast<int>(over) : 0;
    const bool wide = t.flags & kWide;
    float g[8], p[8], m[8], v[8], root[8];
    // the last block of 128 may end before its last lanes: they have zeros
    if (t.flags & kGrad32) load8(static_cast<const float*>(t.grad) + e, wide, left, g);
    else load8(static_cast<const uint16_t*>(t.grad) + e, wide, left, g);
    if (t.master) load8(t.master + e, true, left, p);
    else if (t.flags & kParam32) load8(static_cast<const float*>(t.param) + e, wide, left, p);
    else load8(static_cast<const uint16_t*>(t.param) + e, wide, left, p);
    const int64_t block = e / kAdamwBlock;
    constexpr bool FINE = BITS == 12;
    if (BITS < 32) {
        // codes of whole blocks are there, also past n
        if (base + (threadIdx.x & ~15u) * kEach >= t.n) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = v[i] = 0.0f;
        } else {
            const u32x2 mc = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(t.m) + e);
            const u32x2 vc = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(t.v) + e);
            u32x2 fc = {0, 0};
            if (FINE) fc = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(t.v) + a.fine + e);
            decode8<FINE, 0>(mc, fc, t.m_scale[block], m);
            decode8<FINE, 4>(vc, fc, t.v_scale[block], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * v[i];
        }
    } else {
        load8(static_cast<const float*>(t.m) + e, true, left, m);
        load8(static_cast<const float*>(t.v) + e, true, left, v);
    }
    const float clip = a.grad_scale ? *a.grad_scale : 1.0f;
    if (DEVICE) __syncthreads();
    const Factors f = DEVICE ? shared : a.f;

#pragma unroll
    for (int i = 0; i < 8; ++i) {
        g[i] = g[i] * clip;
        m[i] = m[i] * f.beta1 + g[i] * f.rest1;
        v[i] = v[i] * f.beta2 + (g[i] * g[i]) * f.rest2;
        root[i] = sqrtf(v[i]);
        p[i] = p[i] * f.keep - f.rate * (m[i] / (root[i] * f.root + f.eps));
    }

    if (t.master) save8(t.master + e, true, left, p);
    if (t.flags & kParam32) save8(static_cast<float*>(t.param) + e, wide, left, p);
    else save8(static_cast<uint16_t*>(t.param) + e, wide, left, p);
    if (BITS < 32) {
        // past n the moments are those of zeros
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= left) m[i] = root[i] = 0.0f;
        uint32_t random[8] = {};
        if (FINE) {
            const int64_t number = DEVICE && a.step ? *a.step : a.step_host;
            const uint32_t seed = static_cast<uint32_t>(number) * 0xB5297A4Du + static_cast<uint32_t>(e >> 32) * 0x68E31DA5u;
#pragma unroll
            for (int i = 0; i < 8; ++i) random[i] = dither(static_cast<uint32_t>(e) + i, seed, m[i]);
        }
        u32x2 mc, vc, fc = {0, 0};
        const float ms = encode8<FINE, 0>(m, random, mc, fc), vs = encode8<FINE, 4>(root, random, vc, fc);
        if (base + (threadIdx.x & ~15u) * kEach < t.n) {
            __builtin_nontemporal_store(mc, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(t.m) + e));
            __builtin_nontemporal_store(vc, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(t.v) + e));
            if (FINE) __builtin_nontemporal_store(fc, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(t.v) + a.fine + e));
            if ((threadIdx.x & 15) == 0) {
                t.m_scale[block] = ms;
                t.v_scale[block] = vs;
            }
        }
    } else {
        save8(static_cast<float*>(t.m) + e, true, left, m);
        save8(static_cast<float*>(t.v) + e, true, left, v);
    }
}

hipError_t launch_adamw(const moe_adamw_tensor* tensors, int count, const moe_adamw_hyper& h, int bits,
                        hipStream_t stream) {
    Args a{};
    Factors& f = a.f;
    f.beta1 = static_cast<float>(h.beta1);
    f.rest1 = static_cast<float>(1.0 - h.beta1);
    f.beta2 = static_cast<float>(h.beta2);
    f.rest2 = static_cast<float>(1.0 - h.beta2);
    f.eps = static_cast<float>(h.eps);
    a.log1 = log(h.beta1);
    a.log2 = log(h.beta2);
    a.lr_host = h.lr;
    a.decay = h.weight_decay;
    a.step_host = h.step;
    a.fine = h.fine;
    a.grad_scale = h.grad_scale;
    a.lr = h.lr_device;
    a.step = h.step_device;
    const bool device = a.lr || a.step;
    if (!device) {
        const double t = static_cast<double>(h.step);
        set_rates(f, h.lr, h.weight_decay, bias_fix(a.log1, t), bias_fix(a.log2, t));
    }
    for (int i = 0; i < count;) {
        a.count = 0;
        int64_t blocks = 0;
        for (; i < count && a.count < kAdamwTensors; ++i) {
            const moe_adamw_tensor& s = tensors[i];
            if (s.n == 0) continue;
            Tensor& t = a.t[a.count];
            t = Tensor{s.param, s.grad, s.master, s.m, s.v, s.m_scale, s.v_scale, s.n, 0};
            const uintptr_t both = reinterpret_cast<uintptr_t>(s.param) | reinterpret_cast<uintptr_t>(s.grad);
            t.flags = (s.param_fp32 ? kParam32 : 0) | (s.grad_fp32 ? kGrad32 : 0) | (both % 16 == 0 ? kWide : 0);
            a.first[a.count++] = static_cast<uint32_t>(blocks);
            blocks += (s.n + kAdamwChunk - 1) / kAdamwChunk;
        }
        if (a.count == 0) break;
        const dim3 grid(static_cast<unsigned>(blocks));
        if (bits == 8 && a.fine) {
            if (device) hipLaunchKernelGGL((adamw_kernel<12, true>), grid, dim3(NT), 0, stream, a);
            else hipLaunchKernelGGL((adamw_kernel<12, false>), grid, dim3(NT), 0, stream, a);
        } else if (bits == 8) {
            if (device) hipLaunchKernelGGL((adamw_kernel<8, true>), grid, dim3(NT), 0, stream, a);
            else hipLaunchKernelGGL((adamw_kernel<8, false>), grid, dim3(NT), 0, stream, a);
        } else {
            if (device) hipLaunchKernelGGL((adamw_kernel<32, true>), grid, dim3(NT), 0, stream, a);
            else hipLaunchKernelGGL((adamw_kernel<32, false>), grid, dim3(NT), 0, stream, a);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
