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
    if (c->M > (1 << 19) || c->N > (1 << 19))
        return fail(LA_ERR_UNSUPPORTED, "the backward takes M and N up to 2^19 (M=%d N=%d)", c->M, c->N);
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

}  // extern "C"
