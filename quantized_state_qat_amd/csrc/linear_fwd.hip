// y = s_x s_w (c_x c_w^T) + bias: the product of two matrices of 8-bit codes, exact in 32-bit
// integers, with the scales of tokens (rows) and channels (columns) applied to the sum.
#include "linear_gemm.hpp"

namespace la {
namespace {

// Few tokens: bound by the weights' bytes and, below that, by latency.  A workgroup has 16 channels and
// all tokens (TJ tiles of 16); its eight waves take 128 bytes of the rows in turn, straight into
// registers, and their sums meet in LDS.  M = 1, N = 8192, K = 2048: 512 workgroups whose loads are
// all in flight at once, 5 us with the weights in the caches, 6.1 from memory (tiles of 64 x 64 7.3).
template <class O, int TJ>
__global__ __launch_bounds__(512) void skinny_kernel(GemmArgs a) {
    constexpr int AHEAD = TJ > 2 ? 2 : 4;  // chunks of 128 bytes loaded together
    __shared__ iv4 sums[8][TJ][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int i0 = blockIdx.x * 16;
    const int ni = a.I - i0 < 16 ? a.I - i0 : 16;
    const auto P = make_rsrc(a.P + i0 * a.ldP, (ni - 1) * a.ldP + a.kbytes);
    const auto Q = make_rsrc(a.Q, (a.J - 1) * a.ldQ + a.kbytes);
    const uint32_t po = r * static_cast<uint32_t>(a.ldP) + 32 * q, qo = r * static_cast<uint32_t>(a.ldQ) + 32 * q;
    const uint32_t qn = 16 * static_cast<uint32_t>(a.ldQ);
    const int chunks = (a.kbytes + 127) / 128;
    iv4 acc[TJ] = {};
    for (int c0 = wave; c0 < chunks; c0 += 8 * AHEAD) {
        uv4 p[AHEAD][2], x[AHEAD][2][TJ];
#pragma unroll
        for (int k = 0; k < AHEAD; k++) {
            const int at = (c0 + 8 * k) * 128;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                // past a row's end both operands are zero
                const uint32_t out = at + 32 * q + 16 * h < a.kbytes ? 0 : kOutside;
                p[k][h] = __builtin_bit_cast(uv4, __builtin_amdgcn_raw_buffer_load_b128(P, (po + at + 16 * h) | out, 0, 0));
#pragma unroll
                for (int t = 0; t < TJ; t++)
                    x[k][h][t] = __builtin_bit_cast(uv4, __builtin_amdgcn_raw_buffer_load_b128(Q, (qo + t * qn + at + 16 * h) | out, 0, 0));
            }
        }
#pragma unroll
        for (int k = 0; k < AHEAD; k++)
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int t = 0; t < TJ; t++)
                    acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(iv4, p[k][h]), __builtin_bit_cast(iv4, x[k][h][t]), acc[t], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < TJ; t++) sums[wave][t][lane] = acc[t];
    __syncthreads();
    // result (channel 4 (lane / 16) + v, token 16 t + lane % 16) is element v of lane's sums; channels first
    for (int at = threadIdx.x; at < 256 * TJ; at += 512) {
        const int i = at & 15, j = at >> 4, t = j >> 4;
        if (i >= ni || j >= a.J) continue;
        const int l = 16 * (i >> 2) + (j & 15);
        int s = 0;
#pragma unroll
        for (int w = 0; w < 8; w++) s += reinterpret_cast<const int*>(&sums[w][t][l])[i & 3];
        float v = static_cast<float>(s) * static_cast<const float*>(a.row)[j] * a.col[i0 + i];
        if (a.bias) v += load_elem(a.bias, i0 + i, a.bias_dtype);
        store_elem(a.out, j * a.ldo + i0 + i, sizeof(O) == 2 ? LA_BF16 : LA_F32, v);
    }
}

template <class O>
hipError_t launch(const la_linear_config& c, GemmArgs& g, hipStream_t s) {
    if (c.M <= few_tokens(c.N, c.K)) {
        const unsigned grid = static_cast<unsigned>((c.N + 15) / 16);
        if (c.M <= 16) skinny_kernel<O, 1><<<grid, 512, 0, s>>>(g);
        else if (c.M <= 32) skinny_kernel<O, 2><<<grid, 512, 0, s>>>(g);
        else skinny_kernel<O, 4><<<grid, 512, 0, s>>>(g);
        return hipGetLastError();
    }
    g.part_steps = gemm_steps(g.kbytes, 0);
    return launch_gemm<int8_t, false>(g, cut_forward(c.M, c.N, c.K).tiling, s);
}

}  // namespace

hipError_t launch_linear_fwd(const la_linear_config& c, const LinearArgs& a, hipStream_t s) {
    GemmArgs g;
    g.P = reinterpret_cast<const char*>(a.w), g.Q = reinterpret_cast<const char*>(a.x);
    g.ldP = c.K, g.ldQ = c.ld_x ? c.ld_x : c.K;
    g.I = c.N, g.J = c.M, g.kbytes = c.K;
    g.row = a.xs, g.col = a.ws, g.bias = a.bias, g.bias_dtype = c.w_dtype;
    g.out = a.y, g.out_dtype = c.out_dtype, g.ldo = c.ld_y ? c.ld_y : c.N;
    g.wide = g.ldo * (c.out_dtype == LA_BF16 ? 2 : 4) % 16 == 0;
    return c.out_dtype == LA_BF16 ? launch<uint16_t>(c, g, s) : launch<float>(c, g, s);
}

}  // namespace la
