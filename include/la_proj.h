/*
 * la_proj.h - what stands between two linear recurrences, hand-written HIP for AMD Instinct
 * MI355X (gfx950): the matrix product of 8-bit integer codes with a scale for each token and
 * channel (la_linear_*), and the norms after and before a block, fused with the block's gate,
 * its residual scale and the codes of the next product (la_gate_norm_*).
 *
 * A layer in 8 bits: la_gate_norm_fwd turns the recurrence's output into codes, la_linear_fwd
 * projects them, la_gate_norm_fwd joins the result to the residual stream and emits the codes of
 * the next projection.
 *
 * Conventions are those of la_layer.h: device pointers owned by the caller, 16-byte aligned;
 * nothing allocated, freed or kept past the call; all work on `stream` of the current device;
 * arguments checked on the host before any HIP call; unsupported combinations return
 * LA_ERR_UNSUPPORTED and there is no fallback; thread-safe (a workspace belongs to one call at a
 * time); results do not depend on scheduling.  ld_* is the distance in elements between a tensor's
 * rows, 0 = packed tight.  Outputs and gradients overlap neither inputs nor each other, but where a
 * function says so.
 */
#ifndef LA_PROJ_H
#define LA_PROJ_H

#include "la_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------- matrix product in 8-bit integers with scales */

/*
 * With the codes c_x of M tokens, a scale s_x for each, the codes c_w of N channels and a scale
 * s_w for each (a row of la_norm_fwd's or la_gate_norm_fwd's INT8 output with group 0; a row of
 * weights through the same function with pre = post = 0):
 *     y[m][n] = s_x[m] s_w[n] sum_k c_x[m][k] c_w[n][k] + bias[n].
 * The sum is exact (32-bit integers; codes may be any of -128 .. 127), converted to FP32 and
 * multiplied by s_x and then s_w there.  A NaN or infinity among the scales reaches its row or column.
 */
typedef struct la_linear_config {
    int32_t M, N, K;    /* M and N up to 2^24, with below 2^24 tiles of 64 x 64; K a multiple of 16 up to 65536 */
    int32_t x_dtype;    /* la_dtype of dx */
    int32_t out_dtype;  /* la_dtype of y and dy */
    int32_t w_dtype;    /* la_dtype of bias (its gradient is float32) */
    int32_t dw_dtype;   /* la_dtype of dweight */
    int32_t ld_x;       /* row stride of x_codes, a multiple of 16 (0 = K) */
    int32_t ld_y;       /* row stride of y and dy, any value >= N (0 = N) */
} la_linear_config;

/* x_codes int8 [M][K], x_scales float [M], w_codes int8 [N][K], w_scales float [N], bias [N] or NULL
 * (zeros), y [M][N]. */
la_status la_linear_fwd(const la_linear_config* cfg, const void* x_codes, const float* x_scales, const void* w_codes,
                        const float* w_scales, const void* bias, void* y, void* stream);

/* Gradients for the upstream gradient dy, straight through the codes' rounding, of the values
 * xhat = s_x c_x and what = s_w c_w that they stand for:
 *     dx = dy what ([M][K], tight),   dweight = dy^T xhat ([N][K]),   dbias = the sum of dy's rows (float [N]);
 * each may be NULL.  dy times the scales enters a gradient held in bf16 rounded to FP16's 11 bits (off
 * by at most 2^-11 of the value, an eighth of bf16's own rounding), one held in FP32 as two such parts
 * (2^-22), both under a power of two for its row (for dweight its column): values 2^-29 of the row's
 * largest magnitude or smaller lose more.
 * The codes enter exactly.  Sums are FP32, joined in a fixed order; dbias is summed in double over
 * FP32 sums of 64 rows.  M and N up to 2^19.  Workspace: at least la_linear_bwd_workspace_bytes(cfg) bytes
 * (operands laid out for the products); 0 where there is nothing to sum or the call would be refused. */
la_status la_linear_bwd(const la_linear_config* cfg, const void* x_codes, const float* x_scales, const void* w_codes,
                        const float* w_scales, const void* dy, void* dx, void* dweight, float* dbias, void* workspace,
                        size_t ws_bytes, void* stream);
size_t la_linear_bwd_workspace_bytes(const la_linear_config* cfg);

#ifdef __cplusplus
}
#endif
#endif /* LA_PROJ_H */
