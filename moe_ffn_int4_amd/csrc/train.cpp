// train.cpp -- C entry points of the operators beside the layer's forward (the
// second half of include/moe_int4.h): argument checks and launches. As in api.cpp,
// every check is plain host code that runs before any HIP call.
#include "train.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <memory>
#include <new>

#include "adamw.h"
#include "host.h"
#include "int4.h"

namespace {

using moe::check_ptr;
using moe::fail;

constexpr int64_t kMaxDim = 1 << 20;   // a row of features: 32-bit byte offsets inside a tile
constexpr int64_t kMaxRows = 1 << 30;

int check_width(int64_t v, const char* name) {
    if (v < 8 || v % 8 || v > kMaxDim)
        return fail(MOE_ERR_INVALID_ARG, "%s = %lld must be a multiple of 8 in [8, %lld]", name, (long long)v,
                    (long long)kMaxDim);
    return MOE_OK;
}

int check_rows(int64_t v, const char* name) {
    if (v < 0 || v > kMaxRows)
        return fail(MOE_ERR_INVALID_ARG, "%s = %lld outside [0, 2^30]", name, (long long)v);
    return MOE_OK;
}

int check_act(int32_t act) {
    if (act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH)
        return fail(MOE_ERR_INVALID_ARG, "act %d unknown", act);
    return MOE_OK;
}

struct Span {
    const void* p;
    int64_t bytes;
    const char* name;
};

// an output must not overlap `in`; `same`: it may be that very buffer
int check_apart(const Span& out, const Span& in, bool same = false) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p), b = reinterpret_cast<uintptr_t>(in.p);
    if (!a || !b || (same && a == b && out.bytes == in.bytes)) return MOE_OK;
    if (a < b + static_cast<uintptr_t>(in.bytes) && b < a + static_cast<uintptr_t>(out.bytes))
        return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", out.name, in.name);
    return MOE_OK;
}

int check_product(int64_t P, int64_t E, int64_t N, int64_t K, const int32_t* offsets) {
    CHECK(check_rows(P, "P"));
    if (E < 1 || E > MOE_MAX_EXPERTS)
        return fail(MOE_ERR_INVALID_ARG, "E = %lld outside [1, %d]", (long long)E, MOE_MAX_EXPERTS);
    CHECK(check_width(N, "N"));
    CHECK(check_width(K, "K"));
    if (E * N * K > (1LL << 39)) return fail(MOE_ERR_INVALID_ARG, "weights exceed 1 TiB");
    // the kernels count tiles in 32 bits, also where offsets out of order make every
    // group all P rows
    const int64_t width = N > K ? N : K;
    if (E * (P / 64 + 1) > (1LL << 30) || E * (P / 256 + 1) * (width / 256 + 1) > (1LL << 30))
        return fail(MOE_ERR_INVALID_ARG, "P = %lld with E = %lld and %lld features: too many tiles", (long long)P,
                    (long long)E, (long long)width);
    if (!offsets) {
        if (E != 1) return fail(MOE_ERR_INVALID_ARG, "offsets is NULL with E = %lld", (long long)E);
        return MOE_OK;
    }
    return check_ptr(offsets, "offsets", 4);
}

int run_product(int mode, moe::Epilogue epilogue, const moe::MatmulArgs& a, void* stream) {
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_matmul(mode, epilogue, a, static_cast<hipStream_t>(stream)), "matmul launch");
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_grouped_matmul(const uint16_t* x, const uint16_t* w, const int32_t* offsets, int64_t P, int64_t E,
                       int64_t N, int64_t K, void* y, int32_t out_fp32, void* stream) {
    moe::clear_error();
    CHECK(check_product(P, E, N, K, offsets));
    if (P == 0) return MOE_OK;
    CHECK(check_ptr(x, "x"));
    CHECK(check_ptr(w, "w"));
    CHECK(check_ptr(y, "y"));
    const Span out{y, P * N * (out_fp32 ? 4 : 2), "y"};
    CHECK(check_apart(out, {x, P * K * 2, "x"}));
    CHECK(check_apart(out, {w, E * N * K * 2, "w"}));
    CHECK(check_apart(out, {offsets, (E + 1) * 4, "offsets"}));
    moe::MatmulArgs a{};
    a.a = x;
    a.b = w;
    a.offsets = offsets;
    a.P = P;
    a.E = static_cast<int>(E);
    a.N = N;
    a.K = K;
    a.out = y;
    a.out_fp32 = out_fp32 != 0;
    return run_product(moe::kFwd, moe::Epilogue::kPlain, a, stream);
}

int moe_grouped_matmul_dx(const uint16_t* dy, const uint16_t* w, const int32_t* offsets, int64_t P, int64_t E,
                          int64_t N, int64_t K, void* dx, int32_t out_fp32, void* stream) {
    moe::clear_error();
    CHECK(check_product(P, E, N, K, offsets));
    if (P == 0) return MOE_OK;
    CHECK(check_ptr(dy, "dy"));
    CHECK(check_ptr(w, "w"));
    CHECK(check_ptr(dx, "dx"));
    const Span out{dx, P * K * (out_fp32 ? 4 : 2), "dx"};
    CHECK(check_apart(out, {dy, P * N * 2, "dy"}));
    CHECK(check_apart(out, {w, E * N * K * 2, "w"}));
    CHECK(check_apart(out, {offsets, (E + 1) * 4, "offsets"}));
    moe::MatmulArgs a{};
    a.a = dy;
    a.b = w;
    a.offsets = offsets;
    a.P = P;
    a.E = static_cast<int>(E);
    a.N = N;
    a.K = K;
    a.out = dx;
    a.out_fp32 = out_fp32 != 0;
    return run_product(moe::kDx, moe::Epilogue::kPlain, a, stream);
}

int moe_grouped_matmul_dw(const uint16_t* dy, const uint16_t* x, const int32_t* offsets, int64_t P, int64_t E,
                          int64_t N, int64_t K, void* dw, int32_t out_fp32, int32_t accumulate, void* stream) {
    moe::clear_error();
    CHECK(check_product(P, E, N, K, offsets));
    if (P > 0) {
        CHECK(check_ptr(dy, "dy"));
        CHECK(check_ptr(x, "x"));
    }
    CHECK(check_ptr(dw, "dw"));
    const Span out{dw, E * N * K * (out_fp32 ? 4 : 2), "dw"};
    CHECK(check_apart(out, {dy, P * N * 2, "dy"}));
    CHECK(check_apart(out, {x, P * K * 2, "x"}));
    CHECK(check_apart(out, {offsets, (E + 1) * 4, "offsets"}));
    moe::MatmulArgs a{};
    a.a = dy;
    a.b = x;
    a.offsets = offsets;
    a.P = P;
    a.E = static_cast<int>(E);
    a.N = N;
    a.K = K;
    a.out = dw;
    a.out_fp32 = out_fp32 != 0;
    a.accumulate = accumulate != 0;
    return run_product(moe::kDw, moe::Epilogue::kPlain, a, stream);
}

int moe_linear(const uint16_t* x, const uint16_t* w, const float* bias, int32_t act, const uint16_t* residual,
               int64_t T, int64_t N, int64_t K, void* y, int32_t out_fp32, uint16_t* z, void* stream) {
    moe::clear_error();
    CHECK(check_product(T, 1, N, K, nullptr));
    CHECK(check_act(act));
    if (T == 0) return MOE_OK;
    CHECK(check_ptr(x, "x"));
    CHECK(check_ptr(w, "w"));
    if (bias) CHECK(check_ptr(bias, "bias"));
    if (residual) CHECK(check_ptr(residual, "residual"));
    if (z) CHECK(check_ptr(z, "z"));
    CHECK(check_ptr(y, "y"));
    const Span out{y, T * N * (out_fp32 ? 4 : 2), "y"}, pre{z, T * N * 2, "z"};
    const Span in[4] = {{x, T * K * 2, "x"}, {w, N * K * 2, "w"}, {bias, N * 4, "bias"},
                        {residual, T * N * 2, "residual"}};
    for (int i = 0; i < 4; ++i) {
        CHECK(check_apart(out, in[i], i == 3));
        CHECK(check_apart(pre, in[i]));
    }
    CHECK(check_apart(out, pre));
    moe::MatmulArgs a{};
    a.a = x;
    a.b = w;
    a.P = T;
    a.E = 1;
    a.N = N;
    a.K = K;
    a.out = y;
    a.out_fp32 = out_fp32 != 0;
    a.bias = bias;
    a.residual = residual;
    a.z = z;
    a.act = act;
    return run_product(moe::kFwd, moe::Epilogue::kLinear, a, stream);
}

static int check_int4(int64_t P, int64_t E, int64_t N, int64_t K, int32_t group_size, const int32_t* offsets) {
    if (group_size != 128 && group_size != 64 && group_size != 32)
        return fail(MOE_ERR_INVALID_ARG, "group_size %d unsupported (128, 64 or 32)", group_size);
    if (N < 16 || N % 16) return fail(MOE_ERR_INVALID_ARG, "N = %lld must be a positive multiple of 16", (long long)N);
    if (K < 128 || K % 128)
        return fail(MOE_ERR_INVALID_ARG, "K = %lld must be a positive multiple of 128", (long long)K);
    CHECK(check_product(P, E, N, K, offsets));
    // tiles of 4 rows are counted in 32 bits
    if ((P / 4 + E) * (N / 16) > (1LL << 30))
        return fail(MOE_ERR_INVALID_ARG, "P = %lld with E = %lld and N = %lld: too many tiles", (long long)P, (long long)E,
                    (long long)N);
    return MOE_OK;
}

static int run_int4(const uint16_t* x, const uint8_t* q, const float* scales, const int32_t* offsets, int64_t P, int64_t E,
                    int64_t N, int64_t K, int32_t group_size, void* y, int32_t out_fp32, bool linear,
                    moe::MatmulArgs& m, void* stream) {
    CHECK(check_ptr(x, "x"));
    CHECK(check_ptr(q, "q"));
    CHECK(check_ptr(scales, "scales"));
    CHECK(check_ptr(y, "y"));
    const Span out{y, P * N * (out_fp32 ? 4 : 2), "y"};
    CHECK(check_apart(out, {x, P * K * 2, "x"}));
    CHECK(check_apart(out, {q, E * N * K / 2, "q"}));
    CHECK(check_apart(out, {scales, E * N * (K / group_size) * 4, "scales"}));
    CHECK(check_apart(out, {offsets, (E + 1) * 4, "offsets"}));
    m.a = x;
    m.offsets = offsets;
    m.P = P;
    m.E = static_cast<int>(E);
    m.N = N;
    m.K = K;
    m.out = y;
    m.out_fp32 = out_fp32 != 0;
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_int4(moe::choose_int4(P, E, N, K, group_size), linear, group_size, moe::Int4Args{m, q, scales},
                               static_cast<hipStream_t>(stream)),
              "int4 product launch");
    return MOE_OK;
}

int moe_grouped_matmul_int4(const uint16_t* x, const uint8_t* q, const float* scales, const int32_t* offsets, int64_t P,
                            int64_t E, int64_t N, int64_t K, int32_t group_size, void* y, int32_t out_fp32,
                            void* stream) {
    moe::clear_error();
    CHECK(check_int4(P, E, N, K, group_size, offsets));
    if (P == 0) return MOE_OK;
    moe::MatmulArgs m{};
    return run_int4(x, q, scales, offsets, P, E, N, K, group_size, y, out_fp32, false, m, stream);
}

int moe_linear_int4(const uint16_t* x, const uint8_t* q, const float* scales, const float* bias, int32_t act,
                    const uint16_t* residual, int64_t T, int64_t N, int64_t K, int32_t group_size, void* y,
                    int32_t out_fp32, void* stream) {
    moe::clear_error();
    CHECK(check_int4(T, 1, N, K, group_size, nullptr));
    CHECK(check_act(act));
    if (T == 0) return MOE_OK;
    if (bias) CHECK(check_ptr(bias, "bias"));
    if (residual) CHECK(check_ptr(residual, "residual"));
    const Span out{y, T * N * (out_fp32 ? 4 : 2), "y"};
    CHECK(check_apart(out, {bias, N * 4, "bias"}));
    CHECK(check_apart(out, {residual, T * N * 2, "residual"}, true));
    moe::MatmulArgs m{};
    m.bias = bias;
    m.residual = residual;
    m.act = act;
    return run_int4(x, q, scales, nullptr, T, 1, N, K, group_size, y, out_fp32, true, m, stream);
}

// A gated block's weights: h outputs over d inputs, `twice` for both matrices in one.
static int check_gated(int64_t P, int64_t E, int64_t h, int64_t d, const int32_t* offsets, bool twice) {
    CHECK(check_width(h, "h"));
    if (h > kMaxDim / 2) return fail(MOE_ERR_INVALID_ARG, "h = %lld exceeds %lld", (long long)h, (long long)kMaxDim / 2);
    // the rows of a tile of both matrices are 32-bit byte offsets from its first
    if (twice && (h + 256) * d > (1LL << 31))
        return fail(MOE_ERR_INVALID_ARG, "h = %lld with d = %lld: (h + 256) d exceeds 2^31", (long long)h, (long long)d);
    return check_product(P, E, twice ? 2 * h : h, d, offsets);
}

int moe_gated(const uint16_t* x, const uint16_t* w, const float* bias, const int32_t* offsets, int32_t act, int64_t P,
              int64_t E, int64_t h, int64_t d, uint16_t* y, uint16_t* z, void* stream) {
    moe::clear_error();
    CHECK(check_width(d, "d"));
    CHECK(check_gated(P, E, h, d, offsets, true));
    CHECK(check_act(act));
    if (bias && offsets) return fail(MOE_ERR_INVALID_ARG, "bias with offsets: a dense block alone has one");
    if (P == 0) return MOE_OK;
    CHECK(check_ptr(x, "x"));
    CHECK(check_ptr(w, "w"));
    if (bias) CHECK(check_ptr(bias, "bias"));
    CHECK(check_ptr(y, "y"));
    if (z) CHECK(check_ptr(z, "z"));
    const Span out{y, P * h * 2, "y"}, pre{z, P * h * 4, "z"};
    for (const Span& s : {Span{x, P * d * 2, "x"}, Span{w, E * h * d * 4, "w"}, Span{bias, h * 8, "bias"},
                          Span{offsets, (E + 1) * 4, "offsets"}}) {
        CHECK(check_apart(out, s));
        CHECK(check_apart(pre, s));
    }
    CHECK(check_apart(out, pre));
    moe::MatmulArgs a{};
    a.a = x;
    a.b = w;
    a.offsets = offsets;
    a.P = P;
    a.E = static_cast<int>(E);
    a.N = 2 * h;
    a.K = d;
    a.out = y;
    a.bias = bias;
    a.z = z;
    a.act = act;
    return run_product(moe::kFwd, moe::Epilogue::kGated, a, stream);
}

int moe_gated_dz(const uint16_t* dy, const uint16_t* w2, const uint16_t* z, const int32_t* offsets, int32_t act,
                 int64_t P, int64_t E, int64_t h, int64_t d, uint16_t* dz, uint16_t* y, void* stream) {
    moe::clear_error();
    CHECK(check_width(d, "d"));
    CHECK(check_gated(P, E, h, d, offsets, false));
    CHECK(check_act(act));
    if (P == 0) return MOE_OK;
    CHECK(check_ptr(dy, "dy"));
    CHECK(check_ptr(w2, "w2"));
    CHECK(check_ptr(z, "z"));
    CHECK(check_ptr(dz, "dz"));
    if (y) CHECK(check_ptr(y, "y"));
    const Span out{dz, P * h * 4, "dz"}, again{y, P * h * 2, "y"}, pre{z, P * h * 4, "z"};
    for (const Span& s : {Span{dy, P * d * 2, "dy"}, Span{w2, E * h * d * 2, "w2"}, Span{offsets, (E + 1) * 4, "offsets"}}) {
        CHECK(check_apart(out, s));
        CHECK(check_apart(again, s));
    }
    CHECK(check_apart(out, pre, true));
    CHECK(check_apart(again, pre));
    CHECK(check_apart(out, again));
    moe::MatmulArgs a{};
    a.a = dy;
    a.b = w2;
    a.offsets = offsets;
    a.P = P;
    a.E = static_cast<int>(E);
    a.N = d;
    a.K = h;
    a.out = dz;
    a.gate_z = z;
    a.gate_y = y;
    a.act = act;
    return run_product(moe::kDx, moe::Epilogue::kGatedDz, a, stream);
}

size_t moe_linear_dz_workspace_bytes(int64_t T, int64_t N) {
    if (T < 0 || T > kMaxRows || N < 8 || N % 8 || N > kMaxDim) return 0;
    return static_cast<size_t>(moe::linear_dz_slices(T, N)) * static_cast<size_t>(N) * 4;
}

int moe_linear_dz(const uint16_t* dy, const uint16_t* z, int32_t act, int64_t T, int64_t N, uint16_t* dz,
                  float* db, void* workspace, size_t workspace_bytes, void* stream) {
    moe::clear_error();
    CHECK(check_rows(T, "T"));
    CHECK(check_width(N, "N"));
    CHECK(check_act(act));
    const bool none = act == MOE_ACT_NONE;
    if (none && dz) return fail(MOE_ERR_INVALID_ARG, "dz with act none: it is dy");
    if (none && !db) return fail(MOE_ERR_INVALID_ARG, "act none without db: nothing to compute");
    if (T > 0) {
        CHECK(check_ptr(dy, "dy"));
        if (!none) {
            CHECK(check_ptr(z, "z"));
            CHECK(check_ptr(dz, "dz"));
        }
    }
    const int64_t n = T * N * 2;
    const Span out{dz, n, "dz"}, sums{db, N * 4, "db"};
    CHECK(check_apart(out, {dy, n, "dy"}, true));
    CHECK(check_apart(out, {z, n, "z"}, true));
    if (db) {
        CHECK(check_ptr(db, "db", 4));
        if (!workspace) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
        if (!moe::aligned(workspace, 256)) return fail(MOE_ERR_WORKSPACE, "workspace is not 256-byte aligned");
        const size_t need = moe_linear_dz_workspace_bytes(T, N);
        if (workspace_bytes < need)
            return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
        const Span ws{workspace, static_cast<int64_t>(need), "workspace"};
        for (const Span& s : {Span{dy, n, "dy"}, Span{none ? nullptr : z, n, "z"}, out, ws}) CHECK(check_apart(sums, s));
        for (const Span& s : {Span{dy, n, "dy"}, Span{none ? nullptr : z, n, "z"}, out}) CHECK(check_apart(ws, s));
    }
    if (T == 0 && !db) return MOE_OK;
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_linear_dz(dy, z, act, T, N, dz, db, static_cast<float*>(workspace),
                                    static_cast<hipStream_t>(stream)),
              "linear_dz launch");
    return MOE_OK;
}

int moe_swiglu(const uint16_t* z, int64_t rows, int64_t h, uint16_t* y, void* stream) {
    moe::clear_error();
    CHECK(check_rows(rows, "rows"));
    CHECK(check_width(h, "h"));
    if (rows == 0) return MOE_OK;
    CHECK(check_ptr(z, "z"));
    CHECK(check_ptr(y, "y"));
    CHECK(check_apart({y, rows * h * 2, "y"}, {z, rows * h * 4, "z"}));
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_swiglu(z, rows, h, y, static_cast<hipStream_t>(stream)), "swiglu launch");
    return MOE_OK;
}

int moe_swiglu_backward(const uint16_t* dy, const uint16_t* z, int64_t rows, int64_t h, uint16_t* dz,
                        void* stream) {
    moe::clear_error();
    CHECK(check_rows(rows, "rows"));
    CHECK(check_width(h, "h"));
    if (rows == 0) return MOE_OK;
    CHECK(check_ptr(dy, "dy"));
    CHECK(check_ptr(z, "z"));
    CHECK(check_ptr(dz, "dz"));
    CHECK(check_apart({dz, rows * h * 4, "dz"}, {dy, rows * h * 2, "dy"}));
    CHECK(check_apart({dz, rows * h * 4, "dz"}, {z, rows * h * 4, "z"}, true));
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_swiglu_backward(dy, z, rows, h, dz, static_cast<hipStream_t>(stream)),
              "swiglu_backward launch");
    return MOE_OK;
}

static int check_pairs(int64_t T, int32_t top_k, int64_t d) {
    CHECK(check_rows(T, "T"));
    if (top_k < 1 || top_k > MOE_MAX_TOP_K)
        return fail(MOE_ERR_INVALID_ARG, "top_k = %d outside [1, %d]", top_k, MOE_MAX_TOP_K);
    if (T * top_k > kMaxRows)
        return fail(MOE_ERR_INVALID_ARG, "T * top_k = %lld exceeds 2^30", (long long)(T * top_k));
    return check_width(d, "d");
}

int moe_permute_rows(const uint16_t* x, const int32_t* perm, int64_t T, int32_t top_k, int64_t d, uint16_t* xp,
                     void* stream) {
    moe::clear_error();
    CHECK(check_pairs(T, top_k, d));
    if (T == 0) return MOE_OK;
    CHECK(check_ptr(x, "x"));
    CHECK(check_ptr(perm, "perm", 4));
    CHECK(check_ptr(xp, "xp"));
    const Span out{xp, T * top_k * d * 2, "xp"};
    CHECK(check_apart(out, {x, T * d * 2, "x"}));
    CHECK(check_apart(out, {perm, T * top_k * 4, "perm"}));
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_permute_rows(x, perm, T, top_k, d, xp, static_cast<hipStream_t>(stream)),
              "permute_rows launch");
    return MOE_OK;
}

int moe_combine(const void* o, int32_t o_fp32, const int32_t* inv, const float* gates, const uint16_t* residual,
                int64_t T, int32_t top_k, int64_t d, uint16_t* y, void* stream) {
    moe::clear_error();
    CHECK(check_pairs(T, top_k, d));
    if (T == 0) return MOE_OK;
    CHECK(check_ptr(o, "o"));
    CHECK(check_ptr(inv, "inv", 4));
    if (gates) CHECK(check_ptr(gates, "gates", 4));
    if (residual) CHECK(check_ptr(residual, "residual"));
    CHECK(check_ptr(y, "y"));
    const Span out{y, T * d * 2, "y"};
    CHECK(check_apart(out, {o, T * top_k * d * (o_fp32 ? 4 : 2), "o"}));
    CHECK(check_apart(out, {inv, T * top_k * 4, "inv"}));
    CHECK(check_apart(out, {gates, T * top_k * 4, "gates"}));
    CHECK(check_apart(out, {residual, T * d * 2, "residual"}, true));
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_combine_rows(o, o_fp32 != 0, inv, gates, residual, T, top_k, d, y,
                                       static_cast<hipStream_t>(stream)),
              "combine launch");
    return MOE_OK;
}

int moe_combine_backward(const uint16_t* dy, const void* o, int32_t o_fp32, const int32_t* inv,
                         const float* gates, int64_t T, int32_t top_k, int64_t d, uint16_t* d_o, float* d_gates,
                         void* stream) {
    moe::clear_error();
    CHECK(check_pairs(T, top_k, d));
    if (T == 0) return MOE_OK;
    CHECK(check_ptr(dy, "dy"));
    CHECK(check_ptr(inv, "inv", 4));
    if (gates) CHECK(check_ptr(gates, "gates", 4));
    CHECK(check_ptr(d_o, "d_o"));
    if (d_gates) {
        CHECK(check_ptr(o, "o"));
        CHECK(check_ptr(d_gates, "d_gates", 4));
    }
    const int64_t P = T * top_k;
    const Span rows{d_o, P * d * 2, "d_o"}, sums{d_gates, P * 4, "d_gates"};
    const Span in[4] = {{dy, T * d * 2, "dy"}, {d_gates ? o : nullptr, P * d * (o_fp32 ? 4 : 2), "o"},
                        {inv, P * 4, "inv"}, {gates, P * 4, "gates"}};
    for (const Span& s : in) {
        CHECK(check_apart(rows, s));
        CHECK(check_apart(sums, s));
    }
    CHECK(check_apart(rows, sums));
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_combine_backward(dy, o, o_fp32 != 0, inv, gates, T, top_k, d, d_o, d_gates,
                                           static_cast<hipStream_t>(stream)),
              "combine_backward launch");
    return MOE_OK;
}

// What a step writes must be apart from itself, from every gradient and from the numbers on the device: the
// spans sorted by address, where each need only be apart from those that start before it ends.
static int check_adamw_apart(const moe_adamw_tensor* tensors, int32_t count, const moe_adamw_hyper& hyper, int32_t bits) {
    struct Region {
        uintptr_t from, to;
        const char* name;
        int32_t tensor;  // or -1: of all
        bool written;
    };
    std::unique_ptr<Region[]> all(new (std::nothrow) Region[static_cast<size_t>(count) * 8 + 3]);
    if (!all) return fail(MOE_ERR_INVALID_ARG, "count = %d: no memory for its checks", count);
    size_t n = 0;
    auto put = [&](const void* p, int64_t bytes, const char* name, int32_t tensor, bool written) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p);
        if (p) all[n++] = Region{a, a + static_cast<uintptr_t>(bytes), name, tensor, written};
    };
    put(hyper.step_device, 4, "step_device", -1, false);
    put(hyper.lr_device, 4, "lr_device", -1, false);
    put(hyper.grad_scale, 4, "grad_scale", -1, false);
    for (int32_t i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n == 0) continue;
        const int64_t blocks = (t.n + MOE_ADAMW_BLOCK - 1) / MOE_ADAMW_BLOCK;
        const int64_t moment = bits == 8 ? blocks * MOE_ADAMW_BLOCK : t.n * 4;
        auto add = [&](const void* p, int64_t bytes, const char* name) { put(p, bytes, name, i, true); };
        put(t.grad, t.n * (t.grad_fp32 ? 4 : 2), "grad", i, false);
        add(t.param, t.n * (t.param_fp32 ? 4 : 2), "param");
        add(t.master, t.n * 4, "master");
        add(t.m, moment, "m");
        add(t.v, moment, "v");
        if (bits == 8) {
            add(t.m_scale, blocks * 4, "m_scale");
            add(t.v_scale, blocks * 4, "v_scale");
            if (hyper.fine) add(static_cast<const uint8_t*>(t.v) + hyper.fine, moment, "fine");
        }
    }
    std::sort(all.get(), all.get() + n, [](const Region& a, const Region& b) { return a.from < b.from; });
    const Region *written = nullptr, *read = nullptr;  // those that reach furthest so far
    for (size_t k = 0; k < n; ++k) {
        const Region& r = all[k];
        const Region* other = written && written->to > r.from ? written
                              : r.written && read && read->to > r.from ? read : nullptr;
        if (other) {
            char who[2][48];
            for (int k = 0; k < 2; ++k) {
                const Region& q = k ? *other : r;
                if (q.tensor < 0) snprintf(who[k], sizeof who[k], "%s", q.name);
                else snprintf(who[k], sizeof who[k], "%s of tensor %d", q.name, q.tensor);
            }
            return fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", who[0], who[1]);
        }
        const Region*& most = r.written ? written : read;
        if (!most || r.to > most->to) most = &r;
    }
    return MOE_OK;
}

int moe_adamw(const moe_adamw_tensor* tensors, int32_t count, const moe_adamw_hyper* hyper, int32_t bits,
              void* stream) {
    moe::clear_error();
    if (bits != 8 && bits != 32) return fail(MOE_ERR_INVALID_ARG, "bits = %d: 8 or 32", bits);
    if (count < 0 || count > (1 << 20)) return fail(MOE_ERR_INVALID_ARG, "count = %d outside [0, 2^20]", count);
    if (!hyper) return fail(MOE_ERR_INVALID_ARG, "hyper is NULL");
    if (count > 0 && !tensors) return fail(MOE_ERR_INVALID_ARG, "tensors is NULL");
    const struct {
        double v;
        const char* name;
        bool read;
    } rates[5] = {{hyper->lr, "lr", !hyper->lr_device}, {hyper->beta1, "beta1", true}, {hyper->beta2, "beta2", true},
                  {hyper->eps, "eps", true}, {hyper->weight_decay, "weight_decay", true}};
    for (int i = 0; i < 5; ++i) {
        const bool beta = i == 1 || i == 2;
        if (rates[i].read && !(rates[i].v >= 0 && (beta ? rates[i].v < 1 : std::isfinite(rates[i].v))))
            return fail(MOE_ERR_INVALID_ARG, "%s = %g outside %s", rates[i].name, rates[i].v,
                        beta ? "[0, 1)" : "[0, infinity)");
    }
    if (!hyper->step_device && hyper->step < 1)
        return fail(MOE_ERR_INVALID_ARG, "step = %lld: the first is 1", (long long)hyper->step);
    if (hyper->step_device) CHECK(check_ptr(hyper->step_device, "step_device", 4));
    if (hyper->lr_device) CHECK(check_ptr(hyper->lr_device, "lr_device", 4));
    if (hyper->grad_scale) CHECK(check_ptr(hyper->grad_scale, "grad_scale", 4));
    int64_t all = 0;
    for (int32_t i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n < 0 || t.n > moe::kAdamwMost || (all += t.n) > moe::kAdamwMost)
            return fail(MOE_ERR_INVALID_ARG, "n = %lld of tensor %d: together [0, 2^34]", (long long)t.n, i);
        if (t.n == 0) continue;
        CHECK(check_ptr(t.param, "param", t.param_fp32 ? 4 : 2));
        CHECK(check_ptr(t.grad, "grad", t.grad_fp32 ? 4 : 2));
        if (t.master) CHECK(check_ptr(t.master, "master"));
        CHECK(check_ptr(t.m, "m"));
        CHECK(check_ptr(t.v, "v"));
        if (bits == 8) {
            CHECK(check_ptr(t.m_scale, "m_scale", 4));
            CHECK(check_ptr(t.v_scale, "v_scale", 4));
        } else if (t.m_scale || t.v_scale) {
            return fail(MOE_ERR_INVALID_ARG, "m_scale and v_scale of tensor %d with bits 32", i);
        }
    }
    if (hyper->fine && (bits == 32 || hyper->fine % 16))
        return fail(MOE_ERR_INVALID_ARG, "fine = %lld: a multiple of 16 with bits 8, 0 with bits 32", (long long)hyper->fine);
    if (all == 0) return MOE_OK;
    CHECK(check_adamw_apart(tensors, count, *hyper, bits));
    // codes alone lose every change of less than half their step: with slower moments they stand still
    if (bits == 8 && !hyper->fine && (hyper->beta1 > 0.9 || hyper->beta2 > 0.95))
        return fail(MOE_ERR_INVALID_ARG, "beta1 = %g, beta2 = %g: at most 0.9 and 0.95 for codes alone (fine = 0 with bits 8)",
                    hyper->beta1, hyper->beta2);
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_adamw(tensors, count, *hyper, bits, static_cast<hipStream_t>(stream)), "adamw launch");
    return MOE_OK;
}

}  // extern "C"
