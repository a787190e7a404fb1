// C ABI of the layer operators: argument checks (host only, before any HIP call) and dispatch.
#include "la_check.hpp"

namespace {

la_status check_slots(const int32_t* slots, int32_t n_slots) {
    if (slots && n_slots < 1) return fail(LA_ERR_INVALID_ARG, "n_slots must be >= 1 (n_slots=%d)", n_slots);
    return check_ptr(slots, "slots", false);
}

constexpr int32_t kMaxT = 1 << 30;

// ------------------------------------------------------------------------------ convolution
la_status check_conv(const la_conv_config* c, bool step, bool packed) {
    if (!c) return fail(LA_ERR_INVALID_ARG, "cfg is NULL");
    if (c->B < 0 || c->T < 0 || c->C <= 0)
        return fail(LA_ERR_INVALID_ARG, "negative or zero size (B=%d T=%d C=%d)", c->B, c->T, c->C);
    if (step && c->T != 1) return fail(LA_ERR_INVALID_ARG, "one token needs T == 1 (T=%d)", c->T);
    if (c->C % 8 != 0) return fail(LA_ERR_UNSUPPORTED, "C must be a multiple of 8 (C=%d)", c->C);
    if (c->T > kMaxT) return fail(LA_ERR_UNSUPPORTED, "T must be at most 2^30 (T=%d)", c->T);
    if (c->C > (1 << 20)) return fail(LA_ERR_UNSUPPORTED, "C must be at most 2^20 (C=%d)", c->C);
    if (c->width < 2 || c->width > 4) return fail(LA_ERR_UNSUPPORTED, "width must be 2, 3 or 4 (width=%d)", c->width);
    if (c->act != LA_ACT_NONE && c->act != LA_ACT_SILU) return fail(LA_ERR_INVALID_ARG, "unknown act %d", c->act);
    CHECK(check_dtype(c->x_dtype, "x_dtype"));
    CHECK(check_dtype(c->w_dtype, "w_dtype"));
    CHECK(check_ld(c->ld_x, c->C, c->x_dtype, "ld_x"));
    CHECK(check_ld(c->ld_y, c->C, c->x_dtype, "ld_y"));
    const int64_t tokens = packed ? c->T : static_cast<int64_t>(c->B) * c->T;
    if (tokens * c->C > (int64_t{1} << 36) || static_cast<int64_t>(c->B) * c->C > (int64_t{1} << 32))
        return fail(LA_ERR_UNSUPPORTED, "too many elements (B=%d T=%d C=%d)", c->B, c->T, c->C);
    // The forward's grid stays below 2^32 threads (a larger one is cut short without an error): 16
    // bytes of channels for 16 tokens and for every row of the final states, in two parts of whole
    // workgroups of 256.
    const int64_t lanes = c->C / (c->x_dtype == LA_BF16 ? 8 : 4);
    const int64_t walks = (static_cast<int64_t>(c->T) + 15) / 16 * (packed ? 1 : c->B) + static_cast<int64_t>(c->width - 1) * c->B;
    if (walks * lanes > (int64_t{1} << 32) - 512)
        return fail(LA_ERR_UNSUPPORTED, "too many elements for a grid (B=%d T=%d C=%d)", c->B, c->T, c->C);
    if (c->B > 65535) return fail(LA_ERR_UNSUPPORTED, "B must be <= 65535 (B=%d)", c->B);
    return LA_OK;
}

// ------------------------------------------------------------------------------------- scan
la_status check_scan(const la_scan_config* c, bool step) {
    if (!c) return fail(LA_ERR_INVALID_ARG, "cfg is NULL");
    if (c->B < 0 || c->T < 0 || c->H < 0 || c->G <= 0 || c->d_k <= 0 || c->d_v <= 0)
        return fail(LA_ERR_INVALID_ARG, "negative or zero size (B=%d T=%d H=%d G=%d d_k=%d d_v=%d)", c->B, c->T, c->H,
                    c->G, c->d_k, c->d_v);
    if (c->B > 65535 || c->H > 65535)
        return fail(LA_ERR_UNSUPPORTED, "B and H must each be <= 65535 (B=%d H=%d)", c->B, c->H);
    if (step && c->T != 1) return fail(LA_ERR_INVALID_ARG, "one token needs T == 1 (T=%d)", c->T);
    if (c->H % c->G != 0) return fail(LA_ERR_INVALID_ARG, "G must divide H (H=%d G=%d)", c->H, c->G);
    if (c->d_k != 16 && c->d_k != 32 && c->d_k != 64 && c->d_k != 128)
        return fail(LA_ERR_UNSUPPORTED, "d_k must be 16, 32, 64 or 128 (d_k=%d)", c->d_k);
    if (c->d_v % 64 != 0 || c->d_v > 4096)
        return fail(LA_ERR_UNSUPPORTED, "d_v must be a multiple of 64 up to 4096 (d_v=%d)", c->d_v);
    if (c->softplus != 0 && c->softplus != 1) return fail(LA_ERR_INVALID_ARG, "softplus must be 0 or 1");
    CHECK(check_dtype(c->x_dtype, "x_dtype"));
    CHECK(check_dtype(c->dt_dtype, "dt_dtype"));
    CHECK(check_dtype(c->out_dtype, "out_dtype"));
    CHECK(check_ld(c->ld_x, static_cast<int64_t>(c->H) * c->d_v, c->x_dtype, "ld_x"));
    CHECK(check_ld(c->ld_b, static_cast<int64_t>(c->G) * c->d_k, c->x_dtype, "ld_b"));
    CHECK(check_ld(c->ld_c, static_cast<int64_t>(c->G) * c->d_k, c->x_dtype, "ld_c"));
    if (c->ld_dt != 0 && c->ld_dt < c->H)
        return fail(LA_ERR_INVALID_ARG, "ld_dt = %d is shorter than the row (%d)", c->ld_dt, c->H);
    // byte offsets within 64 rows stay below 2^31
    const int64_t row = static_cast<int64_t>(c->H) * c->d_v;
    if (row > (1 << 23) || c->ld_x > (1 << 23) || c->ld_b > (1 << 23) || c->ld_c > (1 << 23) || c->ld_dt > (1 << 23))
        return fail(LA_ERR_UNSUPPORTED, "rows and row strides must be at most 2^23 elements (H=%d d_v=%d)", c->H, c->d_v);
    if (c->T > kMaxT) return fail(LA_ERR_UNSUPPORTED, "T must be at most 2^30 (T=%d)", c->T);
    // a workgroup a sequence, head and 64 columns
    if (c->B * (row / 64) >= la::kMaxUnits)
        return fail(LA_ERR_UNSUPPORTED, "too many heads: B H d_v / 64 must be below 2^23 (B=%d H=%d d_v=%d)", c->B, c->H, c->d_v);
    return LA_OK;
}
// The backward: a workgroup a chunk and group, a wave a chunk and head.
la_status check_scan_bwd(const la_scan_config* c, bool packed) {
    CHECK(check_scan(c, false));
    if (la::scan_bwd_slots(*c, packed) * c->H >= la::kMaxUnits)
        return fail(LA_ERR_UNSUPPORTED, "too many tokens: the backward takes below 2^23 heads of 64-token chunks (B=%d T=%d H=%d)", c->B, c->T, c->H);
    return LA_OK;
}

// The bytes that la_scan_bwd asks for, of a config that passed the layout's check.  A dense call's
// suffice for a packing too, where a packing of the config is taken at all: one of few or short
// sequences has more chunk slots than they have chunks.
size_t scan_bwd_need(const la_scan_config& c, bool packed) {
    if (c.B == 0 || c.T == 0 || c.H == 0) return 0;  // (zeros only)
    const size_t need = la::scan_bwd_workspace(c, packed);
    if (packed || la::scan_bwd_slots(c, true) * c.H >= la::kMaxUnits) return need;
    const size_t other = la::scan_bwd_workspace(c, true);
    return need > other ? need : other;
}

la_status check_scan_inputs(const void* x, const void* dt, const float* A, const void* b, const void* c, const float* D,
                            const float* bias, bool work) {
    CHECK(check_ptr(x, "x", work));
    CHECK(check_ptr(dt, "dt", work));
    CHECK(check_ptr(A, "A", work));
    CHECK(check_ptr(b, "b", work));
    CHECK(check_ptr(c, "c", work));
    CHECK(check_ptr(D, "D", false));
    return check_ptr(bias, "dt_bias", false);
}

// ------------------------------------------------------------------------------------- norm
la_status check_norm(const la_norm_config* c) {
    if (!c) return fail(LA_ERR_INVALID_ARG, "cfg is NULL");
    if (c->rows < 0 || c->d <= 0) return fail(LA_ERR_INVALID_ARG, "negative or zero size (rows=%d d=%d)", c->rows, c->d);
    if (c->d % 8 != 0 || c->d > 16384)
        return fail(LA_ERR_UNSUPPORTED, "d must be a multiple of 8 up to 16384 (d=%d)", c->d);
    // a row has at most 256 lanes, or one for 4 columns: grids, of whole workgroups of up to 32 rows,
    // stay below 2^32 threads (a larger one is cut short without an error)
    const int64_t lanes = c->d / 4 < 8 ? 8 : c->d / 4 < 256 ? c->d / 4 : 256;
    if ((static_cast<int64_t>(c->rows) + 31) * lanes >= (int64_t{1} << 32)) return fail(LA_ERR_UNSUPPORTED, "too many rows (rows=%d d=%d)", c->rows, c->d);
    if (!(c->eps >= 0.0f)) return fail(LA_ERR_INVALID_ARG, "eps must be >= 0");
    CHECK(check_dtype(c->x_dtype, "x_dtype"));
    CHECK(check_dtype(c->w_dtype, "w_dtype"));
    CHECK(check_dtype(c->out_dtype, "out_dtype"));
    return check_codec(c->qdq, c->group, c->d);
}

}  // namespace

extern "C" {

la_status la_conv_fwd(const la_conv_config* cfg, const int32_t* cu_seqlens, const void* x, const void* weight,
                      const void* bias, const void* state0, void* y, void* state_T, void* stream) {
    CHECK(check_conv(cfg, false, cu_seqlens != nullptr));
    const la_conv_config& c = *cfg;
    const bool work = c.B > 0 && c.T > 0;
    CHECK(check_ptr(cu_seqlens, "cu_seqlens", false));
    CHECK(check_ptr(x, "x", work));
    CHECK(check_ptr(weight, "weight", work));
    CHECK(check_ptr(bias, "bias", false));
    CHECK(check_ptr(state0, "state0", false));
    CHECK(check_ptr(y, "y", work));
    CHECK(check_ptr(state_T, "state_T", false));
    if (state_T && state_T == state0) return fail(LA_ERR_INVALID_ARG, "state_T must not be state0");
    if (c.B == 0) return ok();
    la::ConvArgs a;
    a.cu = cu_seqlens, a.x = x, a.w = weight, a.bias = bias, a.s0 = state0, a.y = y, a.sT = state_T;
    return done(la::launch_conv_fwd(c, a, static_cast<hipStream_t>(stream)), "la_conv_fwd launch");
}

size_t la_conv_bwd_workspace_bytes(const la_conv_config* cfg) {
    if (check_conv(cfg, false, true) != LA_OK) return 0;
    return la::conv_bwd_workspace(*cfg);
}

la_status la_conv_bwd(const la_conv_config* cfg, const int32_t* cu_seqlens, const void* x, const void* weight,
                      const void* bias, const void* state0, const void* dy, const void* dstate_T, void* dx,
                      float* dweight, float* dbias, void* dstate0, void* workspace, size_t ws_bytes, void* stream) {
    CHECK(check_conv(cfg, false, cu_seqlens != nullptr));
    const la_conv_config& c = *cfg;
    const bool work = c.B > 0 && c.T > 0;
    CHECK(check_ptr(cu_seqlens, "cu_seqlens", false));
    CHECK(check_ptr(x, "x", work));
    CHECK(check_ptr(weight, "weight", c.B > 0));
    CHECK(check_ptr(bias, "bias", false));
    CHECK(check_ptr(state0, "state0", false));
    CHECK(check_ptr(dy, "dy", work));
    CHECK(check_ptr(dstate_T, "dstate_T", false));
    CHECK(check_ptr(dx, "dx", work));
    CHECK(check_ptr(dweight, "dweight", true));
    CHECK(check_ptr(dbias, "dbias", false));
    CHECK(check_ptr(dstate0, "dstate0", false));
    CHECK(check_workspace(workspace, ws_bytes, la::conv_bwd_workspace(c)));
    la::ConvArgs a;
    a.cu = cu_seqlens, a.x = x, a.w = weight, a.bias = bias, a.s0 = state0, a.dy = dy, a.dsT = dstate_T, a.dx = dx;
    a.dw = dweight, a.dbias = dbias, a.ds0 = dstate0, a.part = static_cast<float*>(workspace);
    return done(la::launch_conv_bwd(c, a, static_cast<hipStream_t>(stream)), "la_conv_bwd launch");
}

la_status la_conv_step(const la_conv_config* cfg, const void* x, const void* weight, const void* bias, void* state,
                       const int32_t* slots, int32_t n_slots, void* y, void* stream) {
    CHECK(check_conv(cfg, true, false));
    const la_conv_config& c = *cfg;
    const bool work = c.B > 0;
    CHECK(check_slots(slots, n_slots));
    CHECK(check_ptr(x, "x", work));
    CHECK(check_ptr(weight, "weight", work));
    CHECK(check_ptr(bias, "bias", false));
    CHECK(check_ptr(state, "state", work));
    CHECK(check_ptr(y, "y", work));
    if (!work) return ok();
    la::ConvArgs a;
    a.x = x, a.w = weight, a.bias = bias, a.state = state, a.slots = slots, a.n_slots = n_slots, a.y = y;
    return done(la::launch_conv_step(c, a, static_cast<hipStream_t>(stream)), "la_conv_step launch");
}

size_t la_scan_workspace_bytes(const la_scan_config* cfg) {
    if (check_scan(cfg, false) != LA_OK) return 0;
    return la::scan_fwd_workspace(*cfg);
}

la_status la_scan_fwd(const la_scan_config* cfg, const int32_t* cu_seqlens, const void* x, const void* dt,
                      const float* A, const void* b, const void* c, const float* D, const float* dt_bias,
                      const float* S0, void* y, float* S_T, void* workspace, size_t ws_bytes, void* stream) {
    CHECK(check_scan(cfg, false));
    const bool units = cfg->B > 0 && cfg->H > 0;
    const bool work = units && cfg->T > 0;
    CHECK(check_ptr(cu_seqlens, "cu_seqlens", false));
    CHECK(check_scan_inputs(x, dt, A, b, c, D, dt_bias, work));
    CHECK(check_ptr(S0, "S0", false));
    CHECK(check_ptr(y, "y", work));
    CHECK(check_ptr(S_T, "S_T", false));
    if (S_T && S_T == S0) return fail(LA_ERR_INVALID_ARG, "S_T must not be S0");
    CHECK(check_workspace(workspace, ws_bytes, la::scan_fwd_workspace(*cfg)));
    if (!units) return ok();
    la::ScanArgs a;
    a.cu = cu_seqlens, a.x = x, a.dt = dt, a.A = A, a.b = b, a.c = c, a.D = D, a.bias = dt_bias, a.S0 = S0, a.y = y;
    a.ST = S_T, a.ws = static_cast<char*>(workspace);
    return done(la::launch_scan_fwd(*cfg, a, static_cast<hipStream_t>(stream)), "la_scan_fwd launch");
}

size_t la_scan_bwd_workspace_bytes(const la_scan_config* cfg) {
    if (check_scan_bwd(cfg, false) != LA_OK) return 0;
    return scan_bwd_need(*cfg, false);
}

size_t la_scan_bwd_varlen_workspace_bytes(const la_scan_config* cfg) {
    if (check_scan_bwd(cfg, true) != LA_OK) return 0;
    return scan_bwd_need(*cfg, true);
}

la_status la_scan_bwd(const la_scan_config* cfg, const int32_t* cu_seqlens, const void* x, const void* dt,
                      const float* A, const void* b, const void* c, const float* D, const float* dt_bias,
                      const float* S0, const void* dy, const float* dS_T, void* dx, void* ddt, float* dA, void* db,
                      void* dc, float* dD, float* ddt_bias, float* dS0, void* workspace, size_t ws_bytes,
                      void* stream) {
    CHECK(check_scan_bwd(cfg, cu_seqlens != nullptr));
    if (cfg->out_dtype != cfg->x_dtype)
        return fail(LA_ERR_UNSUPPORTED, "the backward takes dy in the inputs' dtype (out_dtype must equal x_dtype)");
    const bool units = cfg->B > 0 && cfg->H > 0;
    const bool work = units && cfg->T > 0;
    CHECK(check_ptr(cu_seqlens, "cu_seqlens", false));
    CHECK(check_scan_inputs(x, dt, A, b, c, D, dt_bias, work));
    CHECK(check_ptr(S0, "S0", false));
    CHECK(check_ptr(dy, "dy", work));
    CHECK(check_ptr(dS_T, "dS_T", false));
    CHECK(check_ptr(dx, "dx", work));
    CHECK(check_ptr(ddt, "ddt", work));
    CHECK(check_ptr(dA, "dA", cfg->H > 0));
    CHECK(check_ptr(db, "db", work));
    CHECK(check_ptr(dc, "dc", work));
    CHECK(check_ptr(dD, "dD", false));
    CHECK(check_ptr(ddt_bias, "ddt_bias", false));
    CHECK(check_ptr(dS0, "dS0", false));
    if (dS0 && dS0 == dS_T) return fail(LA_ERR_INVALID_ARG, "dS0 must not be dS_T");
    CHECK(check_workspace(workspace, ws_bytes, scan_bwd_need(*cfg, cu_seqlens != nullptr)));
    la::ScanArgs a;
    a.cu = cu_seqlens, a.x = x, a.dt = dt, a.A = A, a.b = b, a.c = c, a.D = D, a.bias = dt_bias, a.S0 = S0, a.dy = dy;
    a.dST = dS_T, a.dx = dx, a.ddt = ddt, a.dA = dA, a.db = db, a.dc = dc, a.dD = dD, a.dbias = ddt_bias, a.dS0 = dS0;
    a.ws = static_cast<char*>(workspace);
    return done(la::launch_scan_bwd(*cfg, a, static_cast<hipStream_t>(stream)), "la_scan_bwd launch");
}

la_status la_scan_step(const la_scan_config* cfg, const void* x, const void* dt, const float* A, const void* b,
                       const void* c, const float* D, const float* dt_bias, float* S, const int32_t* slots,
                       int32_t n_slots, void* y, void* stream) {
    CHECK(check_scan(cfg, true));
    const bool work = cfg->B > 0 && cfg->H > 0;
    CHECK(check_slots(slots, n_slots));
    CHECK(check_scan_inputs(x, dt, A, b, c, D, dt_bias, work));
    CHECK(check_ptr(S, "S", work));
    CHECK(check_ptr(y, "y", work));
    if (!work) return ok();
    la::ScanArgs a;
    a.x = x, a.dt = dt, a.A = A, a.b = b, a.c = c, a.D = D, a.bias = dt_bias, a.S = S, a.slots = slots;
    a.n_slots = n_slots, a.y = y;
    return done(la::launch_scan_step(*cfg, a, static_cast<hipStream_t>(stream)), "la_scan_step launch");
}

la_status la_norm_fwd(const la_norm_config* cfg, const void* x, const void* residual, const void* weight, void* res_out,
                      void* y, void* codes, float* scales, void* stream) {
    CHECK(check_norm(cfg));
    const la_norm_config& c = *cfg;
    const bool work = c.rows > 0;
    CHECK(check_ptr(x, "x", work));
    CHECK(check_ptr(residual, "residual", false));
    CHECK(check_ptr(weight, "weight", false));
    CHECK(check_ptr(res_out, "res_out", false));
    CHECK(check_ptr(y, "y", false));
    CHECK(check_ptr(codes, "codes", false));
    CHECK(check_ptr(scales, "scales", false));
    if (c.qdq == LA_QDQ_NONE && (codes || scales))
        return fail(LA_ERR_INVALID_ARG, "codes and scales need a quantizer (cfg->qdq)");
    if (!work) return ok();
    la::NormArgs a;
    a.x = x, a.res = residual, a.w = weight, a.res_out = res_out, a.y = y, a.codes = codes, a.scales = scales;
    return done(la::launch_norm_fwd(c, a, static_cast<hipStream_t>(stream)), "la_norm_fwd launch");
}

size_t la_norm_bwd_workspace_bytes(const la_norm_config* cfg) {
    if (check_norm(cfg) != LA_OK) return 0;
    return la::norm_bwd_workspace(*cfg);
}

la_status la_norm_bwd(const la_norm_config* cfg, const void* h, const void* weight, const void* dy, const void* dres,
                      void* dx, float* dweight, void* workspace, size_t ws_bytes, void* stream) {
    CHECK(check_norm(cfg));
    const la_norm_config& c = *cfg;
    const bool work = c.rows > 0;
    CHECK(check_ptr(h, "h", work));
    CHECK(check_ptr(weight, "weight", false));
    CHECK(check_ptr(dy, "dy", work));
    CHECK(check_ptr(dres, "dres", false));
    CHECK(check_ptr(dx, "dx", work));
    CHECK(check_ptr(dweight, "dweight", false));
    CHECK(check_workspace(workspace, ws_bytes, dweight ? la::norm_bwd_workspace(c) : 0));
    la::NormArgs a;
    a.x = h, a.w = weight, a.dy = dy, a.dres = dres, a.dx = dx, a.dw = dweight, a.part = static_cast<float*>(workspace);
    return done(la::launch_norm_bwd(c, a, static_cast<hipStream_t>(stream)), "la_norm_bwd launch");
}

}  // extern "C"
