// train.cpp -- C entry points of the operators beside the layer's forward (the
// second half of include/moe_int4.h): argument checks and launches. As in api.cpp,
// every check is plain host code that runs before any HIP call.
#include "train.h"

#include "host.h"

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

int run_product(int mode, bool linear, const moe::MatmulArgs& a, void* stream) {
    CHECK(moe::device_ok());
    HIP_CHECK(moe::launch_matmul(mode, linear, a, static_cast<hipStream_t>(stream)), "matmul launch");
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
    return run_product(moe::kFwd, false, a, stream);
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
    return run_product(moe::kDx, false, a, stream);
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
    return run_product(moe::kDw, false, a, stream);
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
    return run_product(moe::kFwd, true, a, stream);
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

}  // extern "C"
