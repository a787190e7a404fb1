// C ABI of the operators between two recurrences: argument checks (host only, before any HIP call)
// and dispatch.
#include "la_check.hpp"
#include "la_proj.hpp"

namespace {

// --------------------------------------------------------------------------- matrix product
int64_t tiles64(int64_t a, int64_t b) { return (a + 63) / 64 * ((b + 63) / 64); }

la_status check_linear(const la_linear_config* c) {
    if (!c) return fail(LA_ERR_INVALID_ARG, "cfg is NULL");
    if (c->M < 0 || c->N < 0 || c->K <= 0)
        return fail(LA_ERR_INVALID_ARG, "negative or zero size (M=%d N=%d K=%d)", c->M, c->N, c->K);
    if (c->K % 16 != 0 || c->K > 65536)
        return fail(LA_ERR_UNSUPPORTED, "K must be a multiple of 16 up to 65536 (K=%d)", c->K);
    // a grid has below 2^32 threads, and at least one workgroup of 256 for 64 x 64 results
    if (c->M > (1 << 24) || c->N > (1 << 24) || tiles64(c->M, c->N) >= (1 << 24))
        return fail(LA_ERR_UNSUPPORTED, "M and N must be at most 2^24, with below 2^24 tiles of 64 x 64 (M=%d N=%d)", c->M, c->N);
    CHECK(check_dtype(c->x_dtype, "x_dtype"));
    CHECK(check_dtype(c->out_dtype, "out_dtype"));
    CHECK(check_dtype(c->w_dtype, "w_dtype"));
    CHECK(check_dtype(c->dw_dtype, "dw_dtype"));
    if (c->ld_x != 0 && c->ld_x < c->K) return fail(LA_ERR_INVALID_ARG, "ld_x = %d is shorter than the row (%d)", c->ld_x, c->K);
    if (c->ld_x % 16 != 0) return fail(LA_ERR_ALIGNMENT, "ld_x = %d is not a multiple of 16 bytes", c->ld_x);
    // byte offsets within 256 rows stay below 2^31
    if (c->ld_x > (1 << 22)) return fail(LA_ERR_UNSUPPORTED, "ld_x must be at most 2^22 (ld_x=%d)", c->ld_x);
    if (c->ld_y != 0 && c->ld_y < c->N) return fail(LA_ERR_INVALID_ARG, "ld_y = %d is shorter than the row (%d)", c->ld_y, c->N);
    return LA_OK;
}
la_status check_linear_bwd(const la_linear_config* c) {
    CHECK(check_linear(c));
    // (a launch lays out 64 x 64 of one or two operands a workgroup, beside the joins of dbias)
    if (c->M > (1 << 19) || c->N > (1 << 19) || tiles64(c->M, c->N) >= (1 << 23))
        return fail(LA_ERR_UNSUPPORTED, "the backward takes M and N up to 2^19, with below 2^23 tiles of 64 x 64 (M=%d N=%d)", c->M, c->N);
    return LA_OK;
}

// ---------------------------------------------------------------------- norms around a block
la_status check_gate(const la_gate_norm_config* c) {
    if (!c) return fail(LA_ERR_INVALID_ARG, "cfg is NULL");
    if (c->rows < 0 || c->d <= 0) return fail(LA_ERR_INVALID_ARG, "negative or zero size (rows=%d d=%d)", c->rows, c->d);
    if (c->d % 8 != 0 || c->d > 16384)
        return fail(LA_ERR_UNSUPPORTED, "d must be a multiple of 8 up to 16384 (d=%d)", c->d);
    // grids, of whole workgroups of up to 32 rows, stay below 2^32 threads (a larger one is cut short without
    // an error)
    const int64_t lanes = la::gate_lanes(c->d);
    if ((static_cast<int64_t>(c->rows) + 31) * lanes >= (int64_t{1} << 32)) return fail(LA_ERR_UNSUPPORTED, "too many rows (rows=%d d=%d)", c->rows, c->d);
    const bool power = c->head >= 16 && c->head <= 512 && (c->head & (c->head - 1)) == 0;
    if (c->head != 0 && !power)
        return fail(LA_ERR_UNSUPPORTED, "head must be 0 (the row), 16, 32, 64, 128, 256 or 512 (head=%d)", c->head);
    if (c->head != 0 && c->d % c->head != 0)
        return fail(LA_ERR_INVALID_ARG, "head must divide d (d=%d head=%d)", c->d, c->head);
    if (!(c->eps >= 0.0f)) return fail(LA_ERR_INVALID_ARG, "eps must be >= 0");
    if (c->gate != LA_GATE_NONE && c->gate != LA_GATE_SILU && c->gate != LA_GATE_SIGMOID)
        return fail(LA_ERR_INVALID_ARG, "unknown gate %d", c->gate);
    if ((c->gate_first & ~1) || (c->post & ~1) || (c->pre & ~1))
        return fail(LA_ERR_INVALID_ARG, "gate_first, post and pre must each be 0 or 1 (%d %d %d)", c->gate_first, c->post, c->pre);
    if (c->gate_first && c->gate == LA_GATE_NONE) return fail(LA_ERR_INVALID_ARG, "gate_first needs a gate");
    CHECK(check_dtype(c->x_dtype, "x_dtype"));
    CHECK(check_dtype(c->w_dtype, "w_dtype"));
    CHECK(check_dtype(c->out_dtype, "out_dtype"));
    CHECK(check_ld(c->ld_x, c->d, c->x_dtype, "ld_x"));
    CHECK(check_ld(c->ld_z, c->d, c->x_dtype, "ld_z"));
    return check_codec(c->qdq, c->group, c->d);
}
la_status check_gate_inputs(const la_gate_norm_config& c, const void* x, const void* z, const void* w_post, const void* alpha,
                            const void* w_pre, bool work) {
    CHECK(check_ptr(x, "x", work));
    CHECK(check_ptr(z, "z", work && c.gate != LA_GATE_NONE));
    if (z && c.gate == LA_GATE_NONE) return fail(LA_ERR_INVALID_ARG, "z needs a gate (cfg->gate)");
    CHECK(check_ptr(w_post, "w_post", false));
    if (w_post && !c.post) return fail(LA_ERR_INVALID_ARG, "w_post needs the norm after the block (cfg->post)");
    CHECK(check_ptr(alpha, "alpha", false));
    CHECK(check_ptr(w_pre, "w_pre", false));
    if (w_pre && !c.pre) return fail(LA_ERR_INVALID_ARG, "w_pre needs the norm before the next block (cfg->pre)");
    return LA_OK;
}

}  // namespace

extern "C" {

la_status la_linear_fwd(const la_linear_config* cfg, const void* x_codes, const float* x_scales, const void* w_codes,
                        const float* w_scales, const void* bias, void* y, void* stream) {
    CHECK(check_linear(cfg));
    const la_linear_config& c = *cfg;
    const bool work = c.M > 0 && c.N > 0;
    CHECK(check_ptr(x_codes, "x_codes", work));
    CHECK(check_ptr(x_scales, "x_scales", work));
    CHECK(check_ptr(w_codes, "w_codes", work));
    CHECK(check_ptr(w_scales, "w_scales", work));
    CHECK(check_ptr(bias, "bias", false));
    CHECK(check_ptr(y, "y", work));
    if (!work) return ok();
    la::LinearArgs a;
    a.x = static_cast<const int8_t*>(x_codes), a.xs = x_scales, a.w = static_cast<const int8_t*>(w_codes), a.ws = w_scales;
    a.bias = bias, a.y = y;
    return done(la::launch_linear_fwd(c, a, static_cast<hipStream_t>(stream)), "la_linear_fwd launch");
}

size_t la_linear_bwd_workspace_bytes(const la_linear_config* cfg) {
    if (check_linear_bwd(cfg) != LA_OK) return 0;
    return la::linear_bwd_workspace(*cfg);
}

la_status la_linear_bwd(const la_linear_config* cfg, const void* x_codes, const float* x_scales, const void* w_codes,
                        const float* w_scales, const void* dy, void* dx, void* dweight, float* dbias, void* workspace,
                        size_t ws_bytes, void* stream) {
    CHECK(check_linear_bwd(cfg));
    const la_linear_config& c = *cfg;
    const bool work = c.M > 0 && c.N > 0;
    CHECK(check_ptr(x_codes, "x_codes", work && dweight));
    CHECK(check_ptr(x_scales, "x_scales", work && dweight));
    CHECK(check_ptr(w_codes, "w_codes", work && dx));
    CHECK(check_ptr(w_scales, "w_scales", work && dx));
    CHECK(check_ptr(dy, "dy", work));
    CHECK(check_ptr(dx, "dx", false));
    CHECK(check_ptr(dweight, "dweight", false));
    CHECK(check_ptr(dbias, "dbias", false));
    CHECK(check_workspace(workspace, ws_bytes, la::linear_bwd_workspace(c)));
    if (!dx && !dweight && !dbias) return ok();
    la::LinearArgs a;
    a.x = static_cast<const int8_t*>(x_codes), a.xs = x_scales, a.w = static_cast<const int8_t*>(w_codes), a.ws = w_scales;
    a.dy = dy, a.dx = dx, a.dw = dweight, a.dbias = dbias, a.work = static_cast<char*>(workspace);
    return done(la::launch_linear_bwd(c, a, static_cast<hipStream_t>(stream)), "la_linear_bwd launch");
}

la_status la_gate_norm_fwd(const la_gate_norm_config* cfg, const void* x, const void* z, const void* w_post, const void* alpha,
                           const void* residual, const void* w_pre, void* h, void* y, void* codes, float* scales,
                           void* stream) {
    CHECK(check_gate(cfg));
    const la_gate_norm_config& c = *cfg;
    const bool work = c.rows > 0;
    CHECK(check_gate_inputs(c, x, z, w_post, alpha, w_pre, work));
    CHECK(check_ptr(residual, "residual", false));
    CHECK(check_ptr(h, "h", false));
    CHECK(check_ptr(y, "y", false));
    CHECK(check_ptr(codes, "codes", false));
    CHECK(check_ptr(scales, "scales", false));
    if (c.qdq == LA_QDQ_NONE && (codes || scales))
        return fail(LA_ERR_INVALID_ARG, "codes and scales need a quantizer (cfg->qdq)");
    if (!work) return ok();
    la::GateArgs a;
    a.x = x, a.z = z, a.w_post = w_post, a.alpha = alpha, a.res = residual, a.w_pre = w_pre, a.h = h, a.y = y;
    a.codes = codes, a.scales = scales;
    return done(la::launch_gate_fwd(c, a, static_cast<hipStream_t>(stream)), "la_gate_norm_fwd launch");
}

size_t la_gate_norm_bwd_workspace_bytes(const la_gate_norm_config* cfg) {
    if (check_gate(cfg) != LA_OK) return 0;
    return la::gate_bwd_workspace(*cfg);
}

la_status la_gate_norm_bwd(const la_gate_norm_config* cfg, const void* x, const void* z, const void* w_post, const void* alpha,
                           const void* h, const void* w_pre, const void* dy, const void* dh, void* dx, void* dz,
                           void* dres, float* dw_post, float* dalpha, float* dw_pre, void* workspace, size_t ws_bytes,
                           void* stream) {
    CHECK(check_gate(cfg));
    const la_gate_norm_config& c = *cfg;
    const bool work = c.rows > 0;
    CHECK(check_gate_inputs(c, x, z, w_post, alpha, w_pre, work));
    CHECK(check_ptr(h, "h", work && c.pre));
    CHECK(check_ptr(dy, "dy", work));
    CHECK(check_ptr(dh, "dh", false));
    CHECK(check_ptr(dx, "dx", work));
    CHECK(check_ptr(dz, "dz", false));
    if (dz && c.gate == LA_GATE_NONE) return fail(LA_ERR_INVALID_ARG, "dz needs a gate (cfg->gate)");
    CHECK(check_ptr(dres, "dres", false));
    CHECK(check_ptr(dw_post, "dw_post", false));
    if (dw_post && !c.post) return fail(LA_ERR_INVALID_ARG, "dw_post needs the norm after the block (cfg->post)");
    CHECK(check_ptr(dalpha, "dalpha", false));
    CHECK(check_ptr(dw_pre, "dw_pre", false));
    if (dw_pre && !c.pre) return fail(LA_ERR_INVALID_ARG, "dw_pre needs the norm before the next block (cfg->pre)");
    CHECK(check_workspace(workspace, ws_bytes, dw_post || dalpha || dw_pre ? la::gate_bwd_workspace(c) : 0));
    la::GateArgs a;
    a.x = x, a.z = z, a.w_post = w_post, a.alpha = alpha, a.w_pre = w_pre, a.h = const_cast<void*>(h), a.dy = dy, a.dh = dh;
    a.dx = dx, a.dz = dz, a.dres = dres, a.dw_post = dw_post, a.dalpha = dalpha, a.dw_pre = dw_pre;
    a.part = static_cast<float*>(workspace);
    return done(la::launch_gate_bwd(c, a, static_cast<hipStream_t>(stream)), "la_gate_norm_bwd launch");
}

}  // extern "C"
