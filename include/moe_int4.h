/*
 * moe_int4.h -- C ABI of the MI355X (gfx950) int4 Mixture-of-Experts
 * feed-forward layer.
 *
 * The layer (discosf.com page "1 卡跑通 Llama 4", section "混合专家路由"):
 * a router scores every expert for each token, the top-k experts are chosen,
 * each chosen expert's SwiGLU FFN runs on its tokens and its output is added
 * back to the token weighted by the token's gate for that expert, and the
 * output of a shared expert that every token passes through is added last.
 * Expert FFN (docs.ifdog.com page "Llama 开源模型系列", section
 * "SwiGLU：门控激活的数学"): (Swish(x W1^T) * (x W3^T)) W2^T with
 * Swish(z) = z * sigmoid(z). Routed-expert weights are int4 in groups of 128
 * (same discosf.com page, section "FP8 / Int4 混合量化"), or of 64 or 32: the
 * smaller group sizes the lshu.cn page expects next (section "维护状态");
 * activations and the shared expert stay bf16 (lshu.cn page, section
 * "量化环节").
 *
 * Conventions for every entry point:
 *   - All data pointers are DEVICE pointers on the current HIP device, owned
 *     by the caller; the library never allocates or frees them and keeps no
 *     pointer after the call returns. `stream` is a hipStream_t (NULL = the
 *     default stream); work is enqueued asynchronously on it.
 *   - bf16 values are passed as uint16_t bit patterns.
 *   - Matrices are row-major. Weights are stored "nt": one row per output
 *     feature, the reduction dimension contiguous (W1, W3: [h, d]; W2: [d, h]).
 *   - Return value: MOE_OK, or an error code; nothing is enqueued when a
 *     validation error is returned. Faults during execution surface at the
 *     caller's next synchronisation. No C++ exception crosses the ABI.
 *     moe_last_error() gives a thread-local detail string for the last error.
 *   - Calls on one stream are ordered; concurrent calls on different streams
 *     must use distinct workspaces.
 */
#ifndef MOE_INT4_H
#define MOE_INT4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_INT4_ABI_VERSION 1

enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,        /* bad shape, null or misaligned pointer */
    MOE_ERR_UNSUPPORTED_DEVICE = 2, /* current device is not gfx950 */
    MOE_ERR_HIP = 3,                /* a HIP runtime call failed */
    MOE_ERR_WORKSPACE = 4           /* workspace missing or too small */
};

enum moe_path {
    MOE_PATH_AUTO = 0,     /* DECODE for at most 64 token-expert pairs; HYBRID when the
                              pairs average under 256 per routed expert; otherwise
                              PREFILL_WIDE */
    MOE_PATH_PREFILL = 1,  /* grouped GEMMs on MFMA for every expert, 128-row tiles */
    MOE_PATH_DECODE = 2,   /* HBM-streaming GEMV over the touched experts */
    MOE_PATH_HYBRID = 3,   /* grouped GEMMs for routed experts with more than 32 pairs
                              (128-row tiles) and for the shared expert (256-row tiles, a
                              launch of its own); routed experts with 1..32 pairs on the
                              streaming kernel, which reads their weights once instead of
                              padding them to GEMM tiles */
    MOE_PATH_PREFILL_WIDE = 4  /* PREFILL with 256 x 256 tiles (one block per CU, twice the
                              MFMA work per fragment read); pays off when experts hold
                              hundreds of rows */
};

/* Limits checked by validation. */
#define MOE_GROUP_SIZE 128     /* the default quantization group; 64 and 32 are also supported */
#define MOE_MAX_EXPERTS 256
#define MOE_MAX_TOP_K 16

/* Static description of an error code; never NULL. */
const char *moe_status_string(int status);

/* Detail text of the last error returned on the calling thread ("" if none). */
const char *moe_last_error(void);

/* MOE_INT4_ABI_VERSION of the built library. */
int moe_abi_version(void);

/* MOE_OK if the current HIP device is a gfx950, else MOE_ERR_UNSUPPORTED_DEVICE
 * (or MOE_ERR_HIP if there is no device). */
int moe_device_check(void);

/*
 * Int4 group quantizer (discosf.com page, section "FP8 / Int4 混合量化",
 * int4_row_quantize). For each group of `group_size` consecutive weights of a
 * row: scale = max(max|w|, 1e-6f) / 8, code = clamp(round_half_even(w / scale),
 * -8, 7), in fp32 with a correctly rounded division.
 *
 *   w       fp32 [rows, K], K % 128 == 0, 16-byte aligned
 *   q       out, uint8 [rows, K/2], 16-byte aligned: byte j of a row holds
 *           code 2j in its low nibble and code 2j+1 in its high nibble, 4-bit
 *           two's complement
 *   scales  out, fp32 [rows, K/group_size]
 *   group_size  128 (MOE_GROUP_SIZE), 64 or 32
 */
int moe_quantize_int4(const float *w, int64_t rows, int64_t K, int32_t group_size,
                      uint8_t *q, float *scales, void *stream);

/*
 * The same quantizer writing the tiled layout the forward pass reads
 * (MI355X-specific storage; codes and scales are bit-identical to
 * moe_quantize_int4, only their order in memory differs). rows % 16 == 0.
 * Tile (rb, g) covers rows 16*rb .. 16*rb+15 and reduction columns
 * 128*g .. 128*g+127; tiles are stored rb-major, t = rb * (K/128) + g. With
 * S = 128 / group_size scales per tile row:
 *   q       byte  t*1024 + ((k % 128)/32)*256 + (row % 16)*16 + (k % 32)/2
 *           (low nibble = even k)
 *   scales  float (t*16 + row % 16)*S + (k % 128)/group_size
 * A wavefront reads one 1 KB tile (and its 64*S B of scales) per access.
 */
int moe_quantize_int4_tiled(const float *w, int64_t rows, int64_t K, int32_t group_size,
                            uint8_t *q, float *scales, void *stream);

/*
 * Repack one matrix quantized by moe_quantize_int4 (the row-major format of
 * the quantizer on the discosf.com page, section "FP8 / Int4 混合量化") into
 * the tiled order moe_forward reads (the layout of moe_quantize_int4_tiled).
 * Bytes and scales move unchanged, so the result is bit-identical to
 * moe_quantize_int4_tiled on the same weights.
 *   q            uint8 [rows, K/2] row-major codes, 16-byte aligned
 *   scales       fp32 [rows, K/group_size] row-major scales
 *   rows         multiple of 16; K multiple of 128; group_size 128, 64 or 32
 *   q_tiled      out, rows*K/2 bytes, 16-byte aligned
 *   scales_tiled out, rows*K/group_size fp32
 * The row-major and tiled buffers must not overlap (MOE_ERR_INVALID_ARG).
 * Asynchronous on `stream`.
 */
int moe_tile_int4(const uint8_t *q, const float *scales, int64_t rows, int64_t K,
                  int32_t group_size, uint8_t *q_tiled, float *scales_tiled, void *stream);

/*
 * Repack a bf16 matrix [rows, K] (rows % 16 == 0, K % 128 == 0) into the
 * tiled order the forward pass reads for the shared expert: tile
 * t = (row/16) * (K/128) + k/128 holds 16 rows x 128 columns as 4 steps of
 * 32 columns, element (row, k) at
 *   t*2048 + ((k % 128)/32)*512 + (row % 16)*32 + (k % 32).
 * src and dst are device buffers of rows*K bf16 and must not overlap.
 */
int moe_pack_bf16_tiled(const uint16_t *src, int64_t rows, int64_t K, uint16_t *dst,
                        void *stream);

typedef struct moe_dims {
    int64_t T;      /* tokens, >= 1 */
    int64_t d;      /* model dim, multiple of 128 */
    int64_t E;      /* routed experts, 1..MOE_MAX_EXPERTS */
    int64_t h;      /* expert hidden dim, multiple of 128 */
    int32_t top_k;  /* 1..min(E, MOE_MAX_TOP_K) */
    int32_t group_size; /* int4 quantization group: 128, 64 or 32 */
} moe_dims;

/* Routed experts, each matrix in the TILED int4 layout: written by
 * moe_quantize_int4_tiled with dims->group_size (g), or by moe_quantize_int4
 * and then moe_tile_int4. Row-major codes passed here are read as tiles and
 * give wrong results (the layouts cannot be told apart from the bytes).
 * Experts are stacked (expert e's matrix starts at e times the matrix size):
 *   w1q, w3q [E] x tiled [h, d]: E*h*d/2 bytes   w1s, w3s: E*h*d/g fp32
 *   w2q      [E] x tiled [d, h]: E*d*h/2 bytes   w2s:      E*d*h/g fp32 */
typedef struct moe_experts_int4 {
    const uint8_t *w1q, *w3q, *w2q;
    const float *w1s, *w3s, *w2s;
} moe_experts_int4;

/* Shared expert, bf16, each matrix packed by moe_pack_bf16_tiled:
 * s1, s3 from [h, d]; s2 from [d, h]. */
typedef struct moe_shared_bf16 {
    const uint16_t *s1, *s3, *s2;
} moe_shared_bf16;

/* Bytes of device workspace moe_forward / moe_route need for `dims`
 * (0 if dims are invalid). */
size_t moe_forward_workspace_bytes(const moe_dims *dims);

/*
 * The MoE feed-forward layer.
 *   x          bf16 [T, d]
 *   router_w   fp32 [E, d]; logit[t,e] = sum_j x[t,j] router_w[e,j] (+ router_b[e])
 *   router_b   fp32 [E] or NULL
 *   experts    routed int4 experts (see moe_experts_int4)
 *   shared     shared bf16 expert
 *   y          out, bf16 [T, d]:
 *              y[t] = shared(x_t) + sum_j gate[t,j] * expert_{id[t,j]}(x_t)
 *   topk_ids   out, int32 [T, top_k] or NULL: chosen experts by descending
 *              logit, ties to the lower id
 *   topk_gates out, fp32 [T, top_k] or NULL: sigmoid of the chosen logits
 *   workspace  device buffer of >= moe_forward_workspace_bytes(dims) bytes,
 *              256-byte aligned; contents are scratch
 * Accumulation is fp32; the only roundings beyond fp32 are the bf16 inputs of
 * the matrix cores (dequantized weights, SwiGLU hidden rows) and the bf16 y.
 */
int moe_forward(const moe_dims *dims, const uint16_t *x, const float *router_w,
                const float *router_b, const moe_experts_int4 *experts,
                const moe_shared_bf16 *shared, uint16_t *y, int32_t *topk_ids,
                float *topk_gates, void *workspace, size_t workspace_bytes,
                void *stream);

/* moe_forward with an explicit path (enum moe_path). */
int moe_forward_path(const moe_dims *dims, const uint16_t *x, const float *router_w,
                     const float *router_b, const moe_experts_int4 *experts,
                     const moe_shared_bf16 *shared, uint16_t *y, int32_t *topk_ids,
                     float *topk_gates, int32_t path, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * moe_forward_path without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc. The workspace is a static device array of
 * MOE_NOALLOC_SCRATCH_BYTES inside the library (each GPU the library runs on
 * holds its own copy until the process ends); nothing is allocated or freed by
 * a call. Layers whose moe_forward_workspace_bytes(dims) exceed it return
 * MOE_ERR_WORKSPACE (64 MiB holds, e.g., up to about 550 tokens at top-1 with
 * d = 5120, h = 8192).
 * The first call on a device does a one-time set-up there (the array's device
 * address and the library's second stream for the hybrid path); make it
 * outside graph capture. Every call on a GPU shares that GPU's array and
 * leaves its contents behind: calls that overlap on one GPU (different
 * streams, or host threads) race on it and must be serialised by the caller.
 * Stage timing (moe_profile_enable) creates events; keep it off here.
 * Arguments, outputs, paths and errors otherwise as moe_forward_path.
 */
#define MOE_NOALLOC_SCRATCH_BYTES (64u << 20)
int moe_forward_noalloc(const moe_dims *dims, const uint16_t *x, const float *router_w,
                        const float *router_b, const moe_experts_int4 *experts,
                        const moe_shared_bf16 *shared, uint16_t *y, int32_t *topk_ids,
                        float *topk_gates, int32_t path, void *stream);

/* Row-wise fp8 (OCP E4M3) quantization of the fp8 routed-expert path: the
 * lshu.cn page (section "量化环节") quantizes each activation row to fp8 with
 * its scale bounded by activation_scale_ub, and holds the weights in fp8 with
 * one scale per row ("FP8 行级", section "三条推理路径差异"). Per row of K
 * values, in fp32 with a correctly rounded division:
 *   scale = min(max(max|v|, 1e-12), ub) / 448,   code = fp8_rne(clamp(v / scale, -448, 448))
 * (no bound for weights; ub <= 0: no bound).
 *
 * moe_quantize_fp8_tiled: weights, w fp32 [rows, K] row-major, rows % 16 == 0,
 *   K % 128 == 0 -> q [rows * K] bytes in the tiled order the forward reads
 *   (tile t = (row/16)*(K/128) + k/128 of 2 KB; byte
 *   t*2048 + ((k%128)/32)*512 + (row%16)*32 + k%32), scales fp32 [rows].
 *   w 16-byte aligned; q and scales 4-byte aligned.
 * moe_quantize_fp8_rows: activations, x bf16 [rows, K] row-major -> q [rows, K]
 *   row-major codes, scales fp32 [rows]. x 8-byte aligned.
 * Both: INVALID_ARG on bad shapes / pointers; asynchronous on `stream`. */
int moe_quantize_fp8_tiled(const float *w, int64_t rows, int64_t K, uint8_t *q, float *scales,
                           void *stream);
int moe_quantize_fp8_rows(const uint16_t *x, int64_t rows, int64_t K, float ub, uint8_t *q,
                          float *scales, void *stream);

/* Routed experts in bf16: the pure-bf16 inference path, which the lshu.cn
 * page "Llama 4 单卡量化推理与选型指南" (section "三条推理路径差异") lists as
 * the accuracy baseline of the int4 and fp8 paths. Each expert's matrix is
 * packed by moe_pack_bf16_tiled and the experts are stacked:
 *   w1, w3 [E] x tiled [h, d]: E*h*d bf16     w2 [E] x tiled [d, h]: E*d*h bf16 */
typedef struct moe_experts_bf16 {
    const uint16_t *w1, *w3, *w2;
} moe_experts_bf16;

/* moe_forward_path with bf16 routed experts: the same layer, workspace, paths,
 * outputs and errors; the routed FFNs use the bf16 weights as given. */
int moe_forward_bf16(const moe_dims *dims, const uint16_t *x, const float *router_w,
                     const float *router_b, const moe_experts_bf16 *experts,
                     const moe_shared_bf16 *shared, uint16_t *y, int32_t *topk_ids,
                     float *topk_gates, int32_t path, void *workspace,
                     size_t workspace_bytes, void *stream);

/* Routed experts in fp8 (OCP E4M3) with one fp32 scale per weight row: the
 * fp8_mixed path of the lshu.cn page "Llama 4 单卡量化推理与选型指南"
 * (sections "三条推理路径差异" and "量化环节"). Each matrix is written by
 * moe_quantize_fp8_tiled and the experts are stacked:
 *   w1q, w3q [E] x tiled [h, d]: E*h*d bytes   w1s, w3s: E*h fp32
 *   w2q      [E] x tiled [d, h]: E*d*h bytes   w2s:      E*d fp32
 * act_ub: the activation scale upper bound (finite, >= 0; 0: no bound). */
typedef struct moe_experts_fp8 {
    const uint8_t *w1q, *w3q, *w2q;
    const float *w1s, *w3s, *w2s;
    float act_ub;
} moe_experts_fp8;

/* Bytes of device workspace moe_forward_fp8 needs for `dims` (0 if invalid):
 * the moe_forward workspace plus the fp8 activation rows and their scales. */
size_t moe_forward_fp8_workspace_bytes(const moe_dims *dims);

/* moe_forward_path with fp8 routed experts. Each routed expert computes, as
 * on the page: x_t quantized per row (moe_quantize_fp8_rows with act_ub);
 * a1 = bf16(xq W1q^T * sx * s1), a3 = bf16(xq W3q^T * sx * s3) (exact fp8
 * products, fp32 sums); h = bf16(silu(a1) a3); h quantized per row the same
 * way; out = bf16(hq W2q^T * sh * s2). The router, the shared bf16 expert,
 * the gates, combine, paths, outputs and errors are those of moe_forward_path;
 * workspace >= moe_forward_fp8_workspace_bytes(dims). */
int moe_forward_fp8(const moe_dims *dims, const uint16_t *x, const float *router_w,
                    const float *router_b, const moe_experts_fp8 *experts,
                    const moe_shared_bf16 *shared, uint16_t *y, int32_t *topk_ids,
                    float *topk_gates, int32_t path, void *workspace,
                    size_t workspace_bytes, void *stream);

/* Bytes of device workspace moe_route alone needs (a prefix of the forward
 * workspace; 0 if dims are invalid; dims->h is ignored). */
size_t moe_route_workspace_bytes(const moe_dims *dims);

/*
 * Routing alone: router logits, top-k + sigmoid gates, and the token->expert
 * dispatch the grouped GEMMs use (discosf.com page, section "混合专家路由").
 * Pairs are p = t * top_k + j. Every output except topk_ids/topk_gates may be
 * NULL.
 *   logits   out, fp32 [T, E] (bias included)
 *   counts   out, int32 [E]: pairs routed to each expert
 *   offsets  out, int32 [E+1]: exclusive prefix sum of counts
 *   perm     out, int32 [T*top_k]: perm[slot] = pair; slots of expert e are
 *            offsets[e]..offsets[e+1]-1, pairs in ascending order
 *   inv      out, int32 [T*top_k]: inv[pair] = slot
 *   workspace >= moe_route_workspace_bytes(dims) bytes, 256-byte aligned
 */
int moe_route(const moe_dims *dims, const uint16_t *x, const float *router_w,
              const float *router_b, int32_t *topk_ids, float *topk_gates,
              float *logits, int32_t *counts, int32_t *offsets, int32_t *perm,
              int32_t *inv, void *workspace, size_t workspace_bytes, void *stream);

/*
 * ------------------------------------------------------------------------
 * Operators beside the forward: a bf16 expert layer's products one by one,
 * with their gradients, for programs that train the layer or put dense layers
 * of their own next to it. They follow the conventions above; all data is bf16
 * unless stated, row-major and 16-byte aligned, with feature widths (N, K, h,
 * d) that are multiples of 8 in [8, 2^20] and row counts in [0, 2^30]. Products
 * and sums are accumulated in fp32 and rounded once, to the output's type, at
 * the end; reduction orders are fixed, so a call on the same inputs gives the
 * same bits. Outputs must not overlap inputs or each other, except where an
 * entry point says that they may be the same buffer (MOE_ERR_INVALID_ARG). NaN
 * and infinities in the inputs propagate as in the formulas, to the outputs
 * whose formula reads them.
 *
 * Except for moe_linear_dz's column sums none needs a workspace, so calls on
 * different streams, and captured graphs of them, share no memory.
 */

/*
 * Activations of moe_linear / moe_linear_dz. They, their slopes and SwiGLU's are
 * evaluated in fp32, before the one rounding of an output: to 2^-19 + |e| 2^-21 of
 * the value (of the larger term, where a slope is a sum of two), e being the exponent
 * in it: z (silu), z^2 / 2 (gelu, whose Phi is a fitted polynomial times exp(-z^2 / 2)),
 * sqrt(8/pi) (z + 0.044715 z^3) (gelu_tanh). Magnitudes below 2^-119 may come out as 0.
 * Past +-90 a slope is its limit, also at infinities.
 */
enum moe_act {
    MOE_ACT_NONE = 0,
    MOE_ACT_RELU = 1,
    MOE_ACT_SILU = 2,      /* z sigmoid(z) */
    MOE_ACT_GELU = 3,      /* z Phi(z), by erf */
    MOE_ACT_GELU_TANH = 4  /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
};

/*
 * Products grouped by expert. Rows offsets[e] .. offsets[e+1] - 1 of the row
 * matrices belong to group e (the `offsets` of moe_route; int32 [E+1] on the
 * device, ascending, within [0, P]); E in [1, MOE_MAX_EXPERTS]; E*N*K at most 2^39,
 * E*P at most about 2^36 and E*P*max(N, K) at most about 2^46 (tiles are counted in
 * 32 bits); more is MOE_ERR_INVALID_ARG.
 * A NULL `offsets` with E = 1 means one group of all P rows (a dense layer).
 *   moe_grouped_matmul:     y[s]  = x[s] W_e^T           x [P, K], w [E, N, K], y [P, N]
 *   moe_grouped_matmul_dx:  dx[s] = dy[s] W_e            dy [P, N], dx [P, K]
 *   moe_grouped_matmul_dw:  dw_e  = sum over the rows s of e of dy[s]^T x[s]
 *                                                        dw [E, N, K]; added to the
 *                           values in dw with `accumulate` (one rounding of the sum)
 * The output is bf16, or fp32 with out_fp32. Groups may be empty: their dw is
 * zero (or unchanged with accumulate). Rows outside every group are not read,
 * and their rows of y and dx are left as they were. Offsets that leave [0, P]
 * or descend are the caller's mistake, which the device alone could see: they are
 * clamped, so that nothing outside the operands is read or written, and which rows
 * of y, dx and dw are then computed is not specified.
 */
int moe_grouped_matmul(const uint16_t *x, const uint16_t *w, const int32_t *offsets,
                       int64_t P, int64_t E, int64_t N, int64_t K, void *y,
                       int32_t out_fp32, void *stream);
int moe_grouped_matmul_dx(const uint16_t *dy, const uint16_t *w, const int32_t *offsets,
                          int64_t P, int64_t E, int64_t N, int64_t K, void *dx,
                          int32_t out_fp32, void *stream);
int moe_grouped_matmul_dw(const uint16_t *dy, const uint16_t *x, const int32_t *offsets,
                          int64_t P, int64_t E, int64_t N, int64_t K, void *dw,
                          int32_t out_fp32, int32_t accumulate, void *stream);

/*
 * Dense layer y = act(x W^T + bias) + residual, one pass: x [T, K], w [N, K],
 * bias fp32 [N] or NULL, residual [T, N] or NULL, y [T, N] bf16 or fp32. With z
 * non-NULL it also writes z = x W^T + bias [T, N] (rounded to bf16; y is computed
 * from the unrounded sum), which moe_linear_dz reads. A bf16 y may be the same
 * buffer as residual.
 */
int moe_linear(const uint16_t *x, const uint16_t *w, const float *bias, int32_t act,
               const uint16_t *residual, int64_t T, int64_t N, int64_t K, void *y,
               int32_t out_fp32, uint16_t *z, void *stream);

/*
 * The gradient of moe_linear through its activation: dz = dy * act'(z) [T, N] and
 * db = the column sums of dz before its rounding, fp32 [N] (NULL: not wanted).
 * relu'(0) = 0. The gradients of x and W are then moe_grouped_matmul_dx /
 * _dw of dz with one group; that of the residual is dy. With act none dz is dy:
 * dz must be NULL, z is not read, and db must be wanted. dz may be the same
 * buffer as dy or z. T = 0 gives db = 0. The workspace (at least
 * moe_linear_dz_workspace_bytes, 256-byte aligned) is needed for db alone.
 */
size_t moe_linear_dz_workspace_bytes(int64_t T, int64_t N);
int moe_linear_dz(const uint16_t *dy, const uint16_t *z, int32_t act, int64_t T, int64_t N,
                  uint16_t *dz, float *db, void *workspace, size_t workspace_bytes,
                  void *stream);

/*
 * Gated block: both up-projections, the activation and the product in one pass, with
 * the gradient back to them. Rows s of group e, as in moe_grouped_matmul (NULL offsets with E = 1: a
 * dense block):
 *   moe_gated:     z[s] = [g | u] = x[s] W_e^T + bias,   y[s] = act(g) u
 *                  x [P, d], w [E, 2h, d]: h gate rows, then the h up rows; bias fp32 [2h] or NULL
 *                  (dense alone); y [P, h]. z [P, 2h] receives g and u, rounded, for the gradient (NULL:
 *                  not wanted; y comes from the unrounded sums).
 *   moe_gated_dz:  dh[s] = dy[s] W2_e,   dz[s] = [dh u act'(g) | dh act(g)]
 *                  dy [P, d] the gradient of the down-projection's output, w2 [E, d, h], z [P, 2h]; dz
 *                  [P, 2h], which may be the same buffer as z; y [P, h] receives act(g) u again, from
 *                  which (with dy) W2's gradient follows (NULL: not wanted). dh is never rounded.
 * The gradients of x and W are then moe_grouped_matmul_dx / _dw of dz with N = 2h, that of bias
 * moe_linear_dz of dz (act none). d and h are multiples of 8, h at most 2^19 and, for
 * moe_gated, (h + 256) d at most 2^31. Rows outside every group are left as they were.
 */
int moe_gated(const uint16_t *x, const uint16_t *w, const float *bias, const int32_t *offsets,
              int32_t act, int64_t P, int64_t E, int64_t h, int64_t d, uint16_t *y, uint16_t *z,
              void *stream);
int moe_gated_dz(const uint16_t *dy, const uint16_t *w2, const uint16_t *z, const int32_t *offsets,
                 int32_t act, int64_t P, int64_t E, int64_t h, int64_t d, uint16_t *dz, uint16_t *y,
                 void *stream);

/*
 * Products with 4-bit weights: moe_grouped_matmul and moe_linear on weights that
 * moe_quantize_int4_tiled (or moe_quantize_int4 and moe_tile_int4) has written, at any
 * number of rows, from a single token on.
 *   moe_grouped_matmul_int4:  y[s] = x[s] (scale * code)_e^T       q [E] x tiled [N, K], scales alike
 *   moe_linear_int4:          y = act(x (scale * code)^T + bias) + residual
 * x [P, K] bf16, y [P, N] bf16 or fp32 with out_fp32; offsets, bias, act and residual as there.
 * N a multiple of 16, K of 128, group_size 128, 64 or 32 (the one it was quantized with). Scales may be any
 * finite numbers. Codes are exact in the products, sums fp32, each group's sum multiplied by its fp32
 * scale: no weight is rounded. A group's sum is formed as that of x (code + 24) less 24 times that of x, so an
 * infinite x gives NaN in its row, and |x| is to stay below 2^110. For the same reason errors go by sum |x scale|, up to 2^-17 of
 * it (measured), and not by sum |x scale code|: one x of 300 among ones, under a code of 0, in a row of codes -1, 0 and 1 leaves an
 * fp32 result 4e-5 of it off, where a product in fp32 is 2e-7 off. A bf16 result's own rounding is 2^-8.
 */
int moe_grouped_matmul_int4(const uint16_t *x, const uint8_t *q, const float *scales,
                            const int32_t *offsets, int64_t P, int64_t E, int64_t N, int64_t K,
                            int32_t group_size, void *y, int32_t out_fp32, void *stream);
int moe_linear_int4(const uint16_t *x, const uint8_t *q, const float *scales, const float *bias,
                    int32_t act, const uint16_t *residual, int64_t T, int64_t N, int64_t K,
                    int32_t group_size, void *y, int32_t out_fp32, void *stream);

/*
 * SwiGLU of rows that hold both up-projections side by side, z = [g | u] [rows, 2h]:
 * y = silu(g) * u [rows, h]; and its gradient dz = [dy u silu'(g) | dy silu(g)]
 * [rows, 2h], which may be the same buffer as z.
 */
int moe_swiglu(const uint16_t *z, int64_t rows, int64_t h, uint16_t *y, void *stream);
int moe_swiglu_backward(const uint16_t *dy, const uint16_t *z, int64_t rows, int64_t h,
                        uint16_t *dz, void *stream);

/*
 * Rows moved between tokens and their experts, by the `perm` and `inv` of
 * moe_route (int32 [T*top_k]; pair = t*top_k + j; top_k in [1, MOE_MAX_TOP_K]).
 *   moe_permute_rows:  xp[s] = x[perm[s] / top_k]        x [T, d], xp [T*top_k, d]
 *   moe_combine:       y[t] = sum_j gates[t, j] o[inv[t, j]] + residual[t]
 *                      o [T*top_k, d] bf16, or fp32 with o_fp32; gates fp32 [T, top_k],
 *                      NULL for 1; residual [T, d] or NULL; y [T, d], which may be the
 *                      same buffer as residual. Without gates it is the gradient of
 *                      moe_permute_rows.
 *   moe_combine_backward:  d_o[inv[t, j]] = gates[t, j] dy[t]      [T*top_k, d] bf16
 *                      d_gates[t, j] = <dy[t], o[inv[t, j]]>        fp32, NULL: not wanted
 *                      (then o is not read)
 * The gradient of residual is dy. An entry of perm or inv outside [0, T*top_k)
 * stands for a row of zeros (its d_gates is 0, and nothing of d_o is written for it).
 * Any entries may repeat in moe_permute_rows and moe_combine; in moe_combine_backward
 * a row of d_o that several entries name holds values of any of them, and one that
 * none names is left as it was.
 */
int moe_permute_rows(const uint16_t *x, const int32_t *perm, int64_t T, int32_t top_k,
                     int64_t d, uint16_t *xp, void *stream);
int moe_combine(const void *o, int32_t o_fp32, const int32_t *inv, const float *gates,
                const uint16_t *residual, int64_t T, int32_t top_k, int64_t d, uint16_t *y,
                void *stream);
int moe_combine_backward(const uint16_t *dy, const void *o, int32_t o_fp32,
                         const int32_t *inv, const float *gates, int64_t T, int32_t top_k,
                         int64_t d, uint16_t *d_o, float *d_gates, void *stream);

/*
 * One AdamW step over many tensors at once, in place, in fp32:
 *   g = grad * grad_scale            m = beta1 m + (1 - beta1) g
 *   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^step) * m / (sqrt(v / (1 - beta2^step)) + eps)
 * p is `master` where it is given, and param is then p rounded; else param itself is read. Products
 * and sums are rounded one by one (no fused multiply-add), except that 1 / sqrt(1 - beta2^step) is a factor.
 *
 * bits 32: m and v are fp32 [n]. bits 8: m and v hold OCP E4M3 codes of m and of sqrt(v) in
 * blocks of MOE_ADAMW_BLOCK elements with a scale each,
 *   most = max(max|x|, 2^-100),   scale = most / 448,   c = x * (448 * (1 / most)),   code = fp8_rne(c),
 * the last block filled up with zeros: m and v have ceil(n / 128) * 128 bytes, m_scale and v_scale
 * ceil(n / 128) floats. What the codes leave is kept beside them, as many bytes again, `fine` bytes behind v:
 * in the low four bits m's, in the high four sqrt(v)'s, a whole number k in [-7, 7],
 *   k = floor((c - code) 14 / s + u),     x = (code + k s / 14) scale,
 * with s the step between codes of code's exponent (2^-9 at least) and u in [0, 1) from a hash of the element's place in its
 * tensor, the step's number and the new m. So a change of any size moves a moment by as much on
 * average, where codes alone, whose step is 1/16 to 1/8 of them, would stay as they are for beta near 1 (v of beta2 = 0.99 for good
 * after gradients fall or rise). The last digits are then random: sqrt(v) has a standard deviation of 1 % for beta2 = 0.95, 2 %
 * for 0.99, 4 % for 0.999 and above (twice that while it falls to a tenth), m one of 0.6 % for beta1 = 0.9, 2 % for 0.99. The
 * same call on the same state gives the same bits. The update takes the moments before they are rounded. All codes, scales and
 * fine bytes 0 are a first step's moments; fine bytes 0 beside codes are those codes.
 * fine = 0: codes alone, for beta1 up to 0.9 and beta2 up to 0.95 (else MOE_ERR_INVALID_ARG). Changes of less than half a code's step
 * are lost. With noisy gradients sqrt(v) of beta2 = 0.95 is within 0.8 and 1.5 of its value in 32 bits for 98 elements of 100, but
 * follows a change more slowly (up to 2.5 times too large 60 steps after gradients fell to a tenth, in those bounds after 200);
 * a gradient that is steady keeps m within 0.6 and 1.1 of its own, and sqrt(v) where it was as long as g^2 / v stays within 0 and 2.2.
 *
 * Types may differ from tensor to tensor. n >= 0; together at most 2^34 elements. param and grad
 * are aligned to their type (16 bytes is faster), all else to 16 bytes. What is written (param,
 * master, m, v, fine bytes and scales of every tensor) must not overlap itself, any gradient or a number that
 * the step reads from the device (MOE_ERR_INVALID_ARG), so a tensor cannot be named twice. A NaN or infinite gradient leaves
 * that element's parameter and moments NaN or infinite (8 bits: an infinite one its whole block's
 * moments); so does a number on the device below 1 to all. A finite one whose square is not, past 1.8e19 after scaling, makes v
 * infinite, so that its parameter stands still from then on (8 bits: its whole block's v). Launches: one for each 52 tensors.
 * No workspace; the tensors' addresses are copied at the call, so that a captured graph steps
 * those tensors again.
 */
#define MOE_ADAMW_BLOCK 128
typedef struct moe_adamw_tensor {
    void *param;        /* bf16 [n], or fp32 with param_fp32 */
    const void *grad;   /* bf16 [n], or fp32 with grad_fp32 */
    float *master;      /* fp32 [n], or NULL */
    void *m, *v;
    float *m_scale, *v_scale; /* bits 8 alone, else NULL */
    int64_t n;
    int32_t param_fp32, grad_fp32;
} moe_adamw_tensor;

typedef struct moe_adamw_hyper {
    double lr, beta1, beta2, eps, weight_decay; /* finite; betas in [0, 1), the rest >= 0 */
    int64_t step;               /* this step's number, 1 for the first; not read with step_device */
    const int32_t *step_device; /* the number on the device, or NULL */
    const float *lr_device;     /* lr on the device (lr is then not read), or NULL */
    const float *grad_scale;    /* on the device, or NULL for 1 */
    int64_t fine;               /* bits 8: bytes from each tensor's v to its fine bytes, a multiple of 16, or 0; else 0 */
} moe_adamw_hyper;

int moe_adamw(const moe_adamw_tensor *tensors, int32_t count, const moe_adamw_hyper *hyper,
              int32_t bits, void *stream);

/*
 * Per-stage timing for benchmarks (not part of the layer's arithmetic).
 * While enabled, each stage of every moe_forward / moe_route call (and each
 * int4 quantizer call, as MOE_STAGE_QUANTIZE) is timed by
 * a pair of hipEvents that its kernels record themselves (hipExtLaunchKernel):
 * at the start of the stage's first kernel and the end of its last, so the
 * time excludes the dispatch gap before the stage. moe_profile_read waits for
 * the recorded events, writes the summed duration in milliseconds and the
 * number of timed stage calls of each stage (arrays of `n` entries,
 * n <= MOE_STAGE_COUNT), and resets the sums. It is off by default; while off,
 * kernels launch plainly (and can be captured in graphs). State is
 * process-wide; it is not meant for concurrent callers.
 */
enum moe_stage {
    MOE_STAGE_ROUTER = 0,      /* K2 router logits */
    MOE_STAGE_TOPK = 1,        /* K2 top-k + gates */
    MOE_STAGE_DISPATCH = 2,    /* K3 */
    MOE_STAGE_UP = 3,          /* K4 + shared up-projection, SwiGLU */
    MOE_STAGE_DOWN = 4,        /* K5 + shared down-projection */
    MOE_STAGE_COMBINE = 5,     /* gate-weighted sum + shared, bf16 out */
    MOE_STAGE_DECODE_UP = 6,   /* decode path: streaming up-projection */
    MOE_STAGE_DECODE_DOWN = 7, /* decode path: streaming down-projection */
    MOE_STAGE_ACT_QUANT = 8,   /* fp8 experts: per-row fp8 quantization of x and H */
    MOE_STAGE_QUANTIZE = 9,    /* K1: moe_quantize_int4 / moe_quantize_int4_tiled calls */
    MOE_STAGE_COUNT = 10
};

/*
 * HBM measurement helpers for benchmarks (not part of the layer's arithmetic):
 * the rates plain streaming reaches on the device, the practical ceiling beside
 * the nominal peak. Device pointers, asynchronous on `stream`; bytes must be a
 * positive multiple of 16 and the pointers 16-byte aligned (MOE_ERR_INVALID_ARG
 * otherwise).
 *   moe_hbm_read: reads every 16-byte word of buf once with the non-temporal
 *     loads of the streaming decode kernels; block b of the launch writes the
 *     XOR of the 32-bit words it read to sink[b] (sink: moe_hbm_read_sink_words()
 *     uint32 words, caller-owned), so the XOR of all sink words is the XOR of
 *     the buffer's words.
 *   moe_hbm_copy: copies bytes from src to dst (buffers must not overlap).
 */
int moe_hbm_read(const void *buf, int64_t bytes, uint32_t *sink, void *stream);
int moe_hbm_read_sink_words(void);
int moe_hbm_copy(void *dst, const void *src, int64_t bytes, void *stream);

int moe_profile_enable(int on);
int moe_profile_read(double *ms, int64_t *launches, int n);
const char *moe_stage_name(int stage);

#ifdef __cplusplus
}
#endif

#endif /* MOE_INT4_H */
