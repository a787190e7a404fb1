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
    int32_t ld_x;       /* row stride of x_codes, a multiple of 16 up to 2^22 (0 = K) */
    int32_t ld_y;       /* row stride of y and dy, any value >= N (0 = N) */
} la_linear_config;

/* x_codes int8 [M][K], x_scales float [M], w_codes int8 [N][K], w_scales float [N], bias [N] or NULL
 * (zeros), y [M][N]. */
la_status la_linear_fwd(const la_linear_config* cfg, const void* x_codes, const float* x_scales, const void* w_codes,
                        const float* w_scales, const void* bias, void* y, void* stream);

/* Gradients for the upstream gradient dy, straight through the codes' rounding, of the values
 * xhat = s_x c_x and what = s_w c_w that they stand for:
 *     dx = dy what ([M][K], tight),   dweight = dy^T xhat ([N][K]),   dbias = the sum of dy's rows (float [N]);
 * each may be NULL.  dy times the scales enters as two FP16 parts of 11 bits (off by at most 2^-22 of the
 * value, whatever the gradient's type) under a power of two for its row (for dweight its column): of values
 * below 2^-17 of the row's largest magnitude up to 2^-39 of that magnitude is lost.
 * dy times a scale is formed in FP32, and must not overflow it.  The codes enter exactly.  Sums are
 * FP32, those of a sum's parts joined in double in a fixed order; dbias is summed in double over FP32 sums of
 * 64 rows.  M and N up to 2^19, with below 2^23 tiles of 64 x 64.  Workspace: at least
 * la_linear_bwd_workspace_bytes(cfg) bytes (operands laid out for both products, whichever gradients are wanted:
 * each is the same, bit for bit, alone and with the others); a query returns 0 where there is nothing to sum
 * and where the call would be refused. */
la_status la_linear_bwd(const la_linear_config* cfg, const void* x_codes, const float* x_scales, const void* w_codes,
                        const float* w_scales, const void* dy, void* dx, void* dweight, float* dbias, void* workspace,
                        size_t ws_bytes, void* stream);
size_t la_linear_bwd_workspace_bytes(const la_linear_config* cfg);

/* ------------------------------------------- norms around a block, its gate and residual scale */

typedef enum { LA_GATE_NONE = 0, LA_GATE_SILU = 1, LA_GATE_SIGMOID = 2 } la_out_gate;

/*
 * Per row of d columns, with act the gate's function and rms(v) = sqrt(mean(v^2) + eps):
 *     u = x act(z)  (gate_first)  or  x
 *     n = u / rms(u) * w_post  (post = 1; over each `head` columns, or over the row)  or  u
 *     p = n  (gate_first or no gate)  or  n act(z)
 *     t = residual + alpha p,      h = t rounded to x_dtype
 *     v = h / rms(h) * w_pre  (pre = 1; over the row)  or  t
 * and, with a quantizer, the codecs of la_norm_fwd on v: y is then the value that a code stands for.  (v of
 * bf16 rows comes from FP32 sums and reciprocal roots, la_norm_fwd's from sums of doubles and quotients: of the
 * formula that both have, post = 0 and pre = 1, codes may differ by one where v is a tie but for its last bits.)
 * post alone is the gated output norm of a recurrence (silu: gated delta rule; sigmoid: per-channel
 * gates; gate_first: state-space layers), post and pre the join of a block's output to the residual
 * stream and the next block's norm; with neither, no gate and no residual, the codes are x's own.
 * Everything is FP32 or wider but h (and y, dx, dz, dres at their types).  Codes and scales are the
 * same for every out_dtype and without y.  NaN and infinities reach what the formula takes them to;
 * codes that stand for NaN are as in la_norm_fwd.
 */
typedef struct la_gate_norm_config {
    int32_t rows, d;    /* d a multiple of 8 up to 16384; (rows + 31) L below 2^32, with L the lanes of a row: 8, 16,
                         * 32, 64, 128, 192, 256 or 384, the first that 8 L >= d holds for, 256 for longer rows */
    int32_t head;       /* columns of one norm after the block: 0 (the row), 16, 32, 64, 128, 256 or 512, dividing d */
    float eps;          /* >= 0 */
    int32_t gate;       /* la_out_gate */
    int32_t gate_first; /* 0 | 1 */
    int32_t post, pre;  /* 0 | 1 */
    int32_t qdq;        /* la_qdq, as in la_norm_config */
    int32_t group;      /* with a quantizer 0 (one scale a row), 16, 32, 64 or 128, dividing d */
    int32_t x_dtype;    /* la_dtype of x, z, residual, h and their gradients */
    int32_t w_dtype;    /* la_dtype of w_post, alpha and w_pre (their gradients are float32) */
    int32_t out_dtype;  /* la_dtype of y and dy */
    int32_t ld_x;       /* row stride of x and dx, a multiple of 16 bytes (0 = d) */
    int32_t ld_z;       /* row stride of z and dz, a multiple of 16 bytes (0 = d) */
} la_gate_norm_config;

/* x [rows][d]; z [rows][d] with a gate, else NULL; w_post [head or d] (post) or NULL (ones); alpha [d] or
 * NULL (ones); residual [rows][d] or NULL (zeros); w_pre [d] (pre) or NULL (ones); h and y [rows][d], codes
 * (int8 or E4M3FN bits [rows][d]) and scales (float [rows][d / group]), each NULL where it is not wanted.
 * h may be residual itself (updated in place); no other overlap. */
la_status la_gate_norm_fwd(const la_gate_norm_config* cfg, const void* x, const void* z, const void* w_post, const void* alpha,
                           const void* residual, const void* w_pre, void* h, void* y, void* codes, float* scales,
                           void* stream);

/* Gradients for the upstream gradients dy (of y; identity straight through the codec and h's rounding)
 * and dh (of h; NULL = zero), from x, z and, with pre, the forward's h (else it may be NULL): dx; dz (with a
 * gate; may be NULL); dres (may be NULL; may be dh itself); dw_post float [head or d] (post), dalpha float
 * [d], dw_pre float [d] (pre), each may be NULL, summed in FP32 over at most 128 rows and beyond in double.
 * Workspace: at least la_gate_norm_bwd_workspace_bytes(cfg) bytes (needed for these three). */
la_status la_gate_norm_bwd(const la_gate_norm_config* cfg, const void* x, const void* z, const void* w_post, const void* alpha,
                           const void* h, const void* w_pre, const void* dy, const void* dh, void* dx, void* dz,
                           void* dres, float* dw_post, float* dalpha, float* dw_pre, void* workspace, size_t ws_bytes,
                           void* stream);
size_t la_gate_norm_bwd_workspace_bytes(const la_gate_norm_config* cfg);

#ifdef __cplusplus
}
#endif
#endif /* LA_PROJ_H */
