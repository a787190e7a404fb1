// y = s_x s_w (c_x c_w^T) + bias: the product of two matrices of 8-bit codes, exact in 32-bit
// integers, with the scales of tokens (rows) and channels (columns) applied to the sum.
#include "linear_gemm.hpp"

namespace la {

hipError_t launch_linear_fwd(const la_linear_config& c, const LinearArgs& a, hipStream_t s) {
    GemmArgs g;
    g.P = reinterpret_cast<const char*>(a.w), g.Q = reinterpret_cast<const char*>(a.x);
    g.ldP = c.K, g.ldQ = c.ld_x ? c.ld_x : c.K;
    g.I = c.N, g.J = c.M, g.kbytes = c.K;
    g.row = a.xs, g.col = a.ws, g.bias = a.bias, g.bias_dtype = c.w_dtype;
    g.out = a.y, g.ldo = c.ld_y ? c.ld_y : c.N;
    g.wide = g.ldo * (c.out_dtype == LA_BF16 ? 2 : 4) % 16 == 0;
    return launch_gemm<int8_t, false>(g, c.out_dtype, s);
}

}  // namespace la
