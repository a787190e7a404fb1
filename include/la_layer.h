/*
 * la_layer.h - operators of the layer around a linear recurrence, hand-written HIP for AMD
 * Instinct MI355X (gfx950): the short causal convolution in front of it (la_conv_*), the
 * selective scan, a recurrence with the same state but no delta correction (la_scan_*), and
 * the RMS norm that adds the residual and can emit 8-bit codes with scales (la_norm_*).
 *
 * Conventions are those of la.h: every tensor pointer is a device pointer owned by the
 * caller, 16-byte aligned; nothing is allocated, freed or kept past the call; all work is
 * enqueued on `stream` (a hipStream_t; NULL = the default stream) of the current device;
 * arguments are checked on the host before any HIP call; unsupported combinations return
 * LA_ERR_UNSUPPORTED and there is no fallback; calls are thread-safe (a workspace belongs to
 * one call at a time); la_last_error() tells what was wrong.  Results do not depend on
 * scheduling: no floating-point atomics.
 *
 * Packed sequences.  cu_seqlens == NULL: B sequences of T tokens, tensors [B][T][...].
 * Otherwise int32 [B + 1] in device memory, non-decreasing from 0 to at most T: sequence b is
 * tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of tensors [T][...], cfg->T the packed length.
 * Boundaries are clamped to [0, T] on the device; decreasing ones are a caller error (results
 * are then unspecified, nothing outside the tensors is touched).  Tokens outside every sequence: their
 * rows of forward outputs are left as they were, their gradients are zero (with B = 0 those of all
 * T tokens, in the gradients that are not NULL).
 *
 * Row strides.  ld_* is the distance in elements between a tensor's rows of consecutive
 * tokens, 0 = packed tight.  The row's own elements are contiguous, rows of [B][T] follow
 * each other at the same distance, and ld_* times the element size is a multiple of 16 bytes:
 * x, b and c of the scan can be the slices of one convolution output, and their gradients
 * the slices of one buffer.
 *
 * Outputs and gradients overlap neither inputs nor each other, but where a function says so.
 */
#ifndef LA_LAYER_H
#define LA_LAYER_H

#include "la.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ short causal convolution */

typedef enum { LA_ACT_NONE = 0, LA_ACT_SILU = 1 } la_act;

/*
 * Depthwise causal convolution of width W over C channels.  With the rows of a sequence
 * preceded by the W - 1 rows of its state, z = state0 ++ x,
 *     pre[t][c] = bias[c] + sum_{j < W} weight[c][j] z[t + j][c],   y = silu(pre) or pre,
 *     state_T   = the last W - 1 rows of z.
 * Sums are FP32 (dweight and dbias over a lane's tokens, joined in double).  B T C (packed: T C) may be up to 2^36 and B C up to 2^32, and, with the tokens'
 * blocks of 16 n = B ceil(T / 16) (packed: ceil(T / 16)), (n + (W - 1) B) C up to 2^32 - 512
 * pieces of 16 bytes.
 */
typedef struct la_conv_config {
    int32_t B, T, C;  /* B up to 65535; T up to 2^30; C a multiple of 8 up to 2^20 */
    int32_t width;    /* 2, 3 or 4 */
    int32_t act;      /* la_act */
    int32_t x_dtype;  /* la_dtype of x, y, the states and their gradients */
    int32_t w_dtype;  /* la_dtype of weight and bias (their gradients are float32) */
    int32_t ld_x;     /* row stride of x and dx (0 = C) */
    int32_t ld_y;     /* row stride of y and dy (0 = C) */
} la_conv_config;

/* weight [C][W]; bias [C] or NULL (zeros); state0 [B][W-1][C], oldest row first, or NULL
 * (zeros); state_T [B][W-1][C] or NULL (not written).  state_T must not overlap state0, nor y
 * the inputs. */
la_status la_conv_fwd(const la_conv_config* cfg, const int32_t* cu_seqlens, const void* x, const void* weight,
                      const void* bias, const void* state0, void* y, void* state_T, void* stream);

/* Gradients for the upstream gradients dy and dstate_T ([B][W-1][C]; NULL = zero): dx, dweight
 * (float [C][W]), dbias (float [C]; may be NULL), dstate0 ([B][W-1][C]; may be NULL).  pre is
 * recomputed from x.  Workspace: at least la_conv_bwd_workspace_bytes(cfg) bytes. */
la_status la_conv_bwd(const la_conv_config* cfg, const int32_t* cu_seqlens, const void* x, const void* weight,
                      const void* bias, const void* state0, const void* dy, const void* dstate_T, void* dx,
                      float* dweight, float* dbias, void* dstate0, void* workspace, size_t ws_bytes, void* stream);
size_t la_conv_bwd_workspace_bytes(const la_conv_config* cfg);

/* One token (cfg->T must be 1): x, y [B][C]; the state is read, shifted by the token and
 * written back in place.  slots == NULL: state [B][W-1][C].  Otherwise entry b's state is
 * state[slots[b]] of a pool [n_slots][W-1][C], with the conventions of la_decode_step_slots:
 * slot 0 and indices outside [0, n_slots) are padding (zero output, no state written), and two
 * live entries must not name one slot. */
la_status la_conv_step(const la_conv_config* cfg, const void* x, const void* weight, const void* bias, void* state,
                       const int32_t* slots, int32_t n_slots, void* y, void* stream);

/* ----------------------------------------------------------------------------- selective scan */

/*
 * Per sequence and head h, with the state S (d_k x d_v) in FP32 and the head's group
 * g = h / (H / G) of b and c:
 *     Delta_t = softplus(dt_t + dt_bias_h)  (softplus = 1)  or  dt_t + dt_bias_h
 *     S_t     = exp(Delta_t A_h) S_{t-1} + Delta_t b_t x_t^T
 *     y_t     = S_t^T c_t + D_h x_t
 * The recurrence of la.h with the scalar gate g = Delta A, k = b, q = c and delta = Delta x.
 * Rates Delta A above zero grow the state; cumulated over 64 tokens they must stay below 88.
 * Steps, decays, states and sums are FP32 or wider.  FP32 inputs meet FP32 products; with bf16 inputs
 * y, dx, db and dc come from operands held to 2^-17 of a value (two bf16 parts), whatever their type,
 * S_T, dS0 and the gradients of dt, A, D and dt_bias from exact ones.
 * An infinity or NaN in x reaches the outputs of its whole block of 64 tokens of the sequence
 * (earlier ones too), as one in dt, b or c those from its own token on, and every later one.
 */
typedef struct la_scan_config {
    int32_t B, T, H, G;    /* B and H up to 65535; T up to 2^30; G divides H */
    int32_t d_k, d_v;      /* d_k 16, 32, 64 or 128; d_v a multiple of 64 up to 4096; H d_v up to 2^23 */
    int32_t softplus;      /* 0 | 1 */
    int32_t x_dtype;       /* la_dtype of x, b, c and their gradients */
    int32_t dt_dtype;      /* la_dtype of dt and ddt */
    int32_t out_dtype;     /* la_dtype of y and dy */
    int32_t ld_x;          /* row strides, up to 2^23, of x and dx (0 = H d_v), */
    int32_t ld_b, ld_c;    /* b and db, c and dc (0 = G d_k), */
    int32_t ld_dt;         /* dt and ddt (0 = H; any value >= H) */
} la_scan_config;

/* x [B][T][H][d_v], dt [B][T][H], b and c [B][T][G][d_k], y [B][T][H][d_v] (tight); A, D,
 * dt_bias float [H] (D and dt_bias may be NULL: zeros); S0, S_T float [B][H][d_k][d_v], each
 * may be NULL (zeros; not written).  S_T must not overlap S0 nor y the inputs.  Workspace: at
 * least la_scan_workspace_bytes(cfg) bytes (0 for many shapes: then NULL will do).
 * B H d_v / 64 must be below 2^23. */
la_status la_scan_fwd(const la_scan_config* cfg, const int32_t* cu_seqlens, const void* x, const void* dt,
                      const float* A, const void* b, const void* c, const float* D, const float* dt_bias,
                      const float* S0, void* y, float* S_T, void* workspace, size_t ws_bytes, void* stream);
size_t la_scan_workspace_bytes(const la_scan_config* cfg);

/* Gradients for the upstream gradients dy and dS_T (NULL = zero): dx, ddt, db, dc laid out and
 * typed as their inputs; dA, dD, ddt_bias float [H] (dD and ddt_bias may be NULL); dS0 (may be
 * NULL).  db and dc are summed over the group's heads (H = 0: zero, where they are not NULL).
 * out_dtype must equal x_dtype.  A call takes below 2^23 heads of 64-token chunks.  Workspace (the
 * state and its gradient at every 64th token, and more): at least la_scan_bwd_workspace_bytes(cfg)
 * bytes; for packed sequences la_scan_bwd_varlen_workspace_bytes(cfg), up to B times less, is
 * enough.  A query returns 0 where the call has nothing to sum (B, T or H = 0) and where it would
 * be refused: the first goes by B sequences of T tokens, the second by a
 * packing of T tokens. */
la_status la_scan_bwd(const la_scan_config* cfg, const int32_t* cu_seqlens, const void* x, const void* dt,
                      const float* A, const void* b, const void* c, const float* D, const float* dt_bias,
                      const float* S0, const void* dy, const float* dS_T, void* dx, void* ddt, float* dA, void* db,
                      void* dc, float* dD, float* ddt_bias, float* dS0, void* workspace, size_t ws_bytes,
                      void* stream);
size_t la_scan_bwd_workspace_bytes(const la_scan_config* cfg);
size_t la_scan_bwd_varlen_workspace_bytes(const la_scan_config* cfg);

/* One token (cfg->T must be 1): the state is updated in place.  slots and n_slots as in
 * la_conv_step, over a pool float [n_slots][H][d_k][d_v]. */
la_status la_scan_step(const la_scan_config* cfg, const void* x, const void* dt, const float* A, const void* b,
                       const void* c, const float* D, const float* dt_bias, float* S, const int32_t* slots,
                       int32_t n_slots, void* y, void* stream);

/* -------------------------------------------------- RMS norm with the residual's addition */

/*
 * Per row:  h = x + residual, rounded to x_dtype (what res_out holds and the norm reads),
 *     n = h / sqrt(mean(h^2) + eps) * weight    in FP32,
 * and, with a quantizer, per group of `group` consecutive columns (0 = the whole row) the
 * codecs of la.h on n:  INT8 s = amax/127, code = clamp(rne(n/s), -127, 127);  E4M3 s =
 * amax/448, code = e4m3(n/s)  (s = 1 when amax == 0);  y is then the value the code stands
 * for, code * s (n / s within FP32's rounding of the middle between two codes may take either).
 * Codes and scales are the same for every out_dtype and without y.
 * A row with an infinity or NaN among its h gives NaN where the formula does: in y, and with a
 * quantizer in the scale and every y of a group that holds one.  Codes that stand for NaN are 0
 * (INT8) or NaN (E4M3).
 */
typedef struct la_norm_config {
    int32_t rows, d;    /* (rows + 31) min(256, max(8, d / 4)) below 2^32; d a multiple of 8 up to 16384 */
    float eps;          /* >= 0 */
    int32_t qdq;        /* la_qdq: LA_QDQ_NONE, LA_QDQ_INT8_GROUP or LA_QDQ_E4M3_TILE (one row high) */
    int32_t group;      /* with a quantizer 0, 16, 32, 64 or 128, dividing d */
    int32_t x_dtype;    /* la_dtype of x, residual, res_out and their gradients */
    int32_t w_dtype;    /* la_dtype of weight (its gradient is float32) */
    int32_t out_dtype;  /* la_dtype of y and dy */
} la_norm_config;

/* x [rows][d]; residual [rows][d] or NULL (zeros); weight [d] or NULL (ones); res_out, y and,
 * with a quantizer, codes (int8 or E4M3FN bits [rows][d]) and scales (float [rows][d / group]),
 * each NULL where it is not wanted (codes without scales or the reverse too).  res_out may be
 * residual or x itself (updated in place); no other overlap. */
la_status la_norm_fwd(const la_norm_config* cfg, const void* x, const void* residual, const void* weight, void* res_out,
                      void* y, void* codes, float* scales, void* stream);

/* Gradients for the upstream gradients dy (of y; identity straight through the codec) and
 * dres (of res_out; NULL = zero) from h = the forward's res_out: dx [rows][d] is the gradient
 * of x and of residual alike; dweight float [d] (may be NULL).  dx may be dres itself.
 * Workspace: at least la_norm_bwd_workspace_bytes(cfg) bytes. */
la_status la_norm_bwd(const la_norm_config* cfg, const void* h, const void* weight, const void* dy, const void* dres,
                      void* dx, float* dweight, void* workspace, size_t ws_bytes, void* stream);
size_t la_norm_bwd_workspace_bytes(const la_norm_config* cfg);

#ifdef __cplusplus
}
#endif
#endif /* LA_LAYER_H */
