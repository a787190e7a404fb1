// Norms around a block with its gate and residual scale:
//     u = x act(z) (gate first) or x,   n = u / rms(u over a head or the row) * w_post,
//     p = n act(z) (gate last) or n,    t = residual + alpha p,   h = rne(t),
//     v = h / rms(h) * w_pre  or t,     and 8-bit codes of v,
// and its backward.  Memory bound: one pass over the data, a row in the registers of 8 to 256 lanes
// (1024 in the backward) between its loads, its two norms and its outputs, as in the residual norm.
// A head of 16 to 512 columns is 2 to 64 neighbouring lanes, whose sum needs no LDS.
#include "la_norm.hpp"
#include "la_proj.hpp"

namespace la {
namespace {

// Sum over aligned groups of `n` lanes (a power of two up to 64, the same for the whole launch).
__device__ __forceinline__ float sum_lanes(float x, int n) {
    if (n >= 2) x = x + dpp<kDppXor1>(x);
    if (n >= 4) x = x + dpp<kDppXor2>(x);
    if (n >= 8) x = x + dpp<kDppHalfMirror>(x);
    if (n >= 16) x = x + dpp<kDppMirror>(x);
    if (n >= 32) { Pair p = swap16(x); x = p.a + p.b; }
    if (n >= 64) { Pair p = swap32(x); x = p.a + p.b; }
    return x;
}
__device__ __forceinline__ double sum_lanes(double x, int n) {
    if (n >= 2) x += dpp_double<kDppXor1>(x);
    if (n >= 4) x += dpp_double<kDppXor2>(x);
    if (n >= 8) x += dpp_double<kDppHalfMirror>(x);
    if (n >= 16) x += dpp_double<kDppMirror>(x);
    if (n >= 32) x += __shfl_xor(x, 16);
    if (n >= 64) x += __shfl_xor(x, 32);
    return x;
}
// Sum over the row's lanes, in one barrier: `lds` belongs to this call alone.
template <int LANES, class S>
__device__ __forceinline__ S sum_row(S x, S* lds) {
    x = sum_lanes(x, LANES < 64 ? LANES : 64);
    if constexpr (LANES <= 64) return x;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    S s = lds[0];
#pragma unroll
    for (int k = 1; k < LANES / 64; k++) s += lds[k];
    return s;
}

// act(z), and its derivative.
template <class T>
__device__ __forceinline__ float gate_of(float z, int gate) {
    const float s = sigmoid_for<T>(z);
    return gate == LA_GATE_SILU ? (z < -89.0f ? 0.0f : z * s) : s;
}
template <class T>
__device__ __forceinline__ void gate_both(float z, int gate, float& g, float& slope) {
    const float s = sigmoid_for<T>(z);
    if (gate == LA_GATE_SILU) {
        g = z < -89.0f ? 0.0f : z * s;  // (s is 0 there: of z = -inf too)
        slope = z < -89.0f ? 0.0f : s * (1.0f + z * (1.0f - s));
    } else {
        g = s;
        slope = s * (1.0f - s);
    }
}

struct GateFwd {
    int rows, d, head, gate, first, post, pre, group, w_dtype;
    float eps;
    int64_t ld_x, ld_z;
    const void* x;
    const void* z;
    const void* w_post;
    const void* alpha;
    const void* res;
    const void* w_pre;
    void* h;
    void* y;
    uint8_t* codes;
    float* scales;
};

template <class T, class O, int LANES, int CH, int QDQ>
__global__ __launch_bounds__(256) void gate_fwd_kernel(GateFwd p) {
    constexpr int RPW = 256 / LANES;
    // With codes every operation is rounded as the formula has it and squares are summed in double (as
    // in the residual norm): codes do not depend on y's type or on whether y is wanted.  Their gate is
    // the finer one whatever the type.
    constexpr bool STEPWISE = QDQ != LA_QDQ_NONE;
    typedef std::conditional_t<STEPWISE, double, float> S;
    typedef std::conditional_t<STEPWISE, float, T> G;
    __shared__ S sums[2][4];
    __shared__ float lds[8];
    const int l = threadIdx.x % LANES;
    const int row = blockIdx.x * RPW + threadIdx.x / LANES;
    if (LANES <= 64 && row >= p.rows) return;  // whole groups of lanes leave together
    const size_t base = static_cast<size_t>(row) * p.d;
    const T* x = static_cast<const T*>(p.x) + row * p.ld_x;
    const T* z = p.z ? static_cast<const T*>(p.z) + row * p.ld_z : nullptr;
    float t[CH][8], g[CH][8], r[CH][8];
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int col = (c * LANES + l) * kPiece;
#pragma unroll
        for (int e = 0; e < 8; e++) t[c][e] = r[c][e] = 0.0f, g[c][e] = 1.0f;
        if (col < p.d) {
            load8(x + col, t[c]);
            if (z) load8(z + col, g[c]);
            if (p.res) load8(static_cast<const T*>(p.res) + base + col, r[c]);
        }
    }
    if (z) {
#pragma unroll
        for (int c = 0; c < CH; c++)
#pragma unroll
            for (int e = 0; e < 8; e++) g[c][e] = gate_of<G>(g[c][e], p.gate);
        if (p.first) {
#pragma unroll
            for (int c = 0; c < CH; c++)
#pragma unroll
                for (int e = 0; e < 8; e++) t[c][e] *= g[c][e];
        }
    }
    // v / rms: stepwise by the correctly rounded quotient, else by the reciprocal root
    auto unit = [](float (&v)[8], S sum, int n, float eps) {
        if constexpr (STEPWISE) {
            const float rms = sqrtf(static_cast<float>(sum / n) + eps);
            const bool fast = rms > 0x1p-60f && rms < 0x1p60f;
            const float e0 = __builtin_amdgcn_rcpf(rms);
            const float recip = __builtin_fmaf(__builtin_fmaf(-rms, e0, 1.0f), e0, e0);
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = fast ? quot_rn_fast(v[e], rms, recip) : v[e] / rms;
        } else {
            const float k = rsqrt_fine(static_cast<float>(sum) / static_cast<float>(n) + eps);
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] *= k;
        }
    };
    auto squares = [](const float (&v)[8]) {
        S s = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if constexpr (STEPWISE) s += v[e] * v[e];
            else s = __builtin_fmaf(v[e], v[e], s);
        }
        return s;
    };
    if (p.post) {
        S row_ss = 0;
        if (p.head == 0) {
#pragma unroll
            for (int c = 0; c < CH; c++) row_ss += squares(t[c]);
            row_ss = sum_row<LANES>(row_ss, sums[0]);
        }
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            const S ss = p.head ? sum_lanes(squares(t[c]), p.head / kPiece) : row_ss;
            unit(t[c], ss, p.head ? p.head : p.d, p.eps);
            float w[8];
            if (p.w_post && col < p.d) {
                load_w(p.w_post, p.w_dtype, p.head ? col & (p.head - 1) : col, w);
#pragma unroll
                for (int e = 0; e < 8; e++) t[c][e] *= w[e];
            }
        }
    }
    S ss = 0;
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int col = (c * LANES + l) * kPiece;
        if (col >= p.d) {
#pragma unroll
            for (int e = 0; e < 8; e++) t[c][e] = 0.0f;
            continue;
        }
        if (z && !p.first) {
#pragma unroll
            for (int e = 0; e < 8; e++) t[c][e] *= g[c][e];
        }
        if (p.alpha) {
            float w[8];
            load_w(p.alpha, p.w_dtype, col, w);
#pragma unroll
            for (int e = 0; e < 8; e++) t[c][e] *= w[e];
        }
        if (p.res) {
#pragma unroll
            for (int e = 0; e < 8; e++) t[c][e] += r[c][e];
        }
        if (p.h) store8(static_cast<T*>(p.h) + base + col, t[c]);
        if (p.pre) {  // the norm reads what h holds
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const uint32_t u = pack16(t[c][e], t[c][e + 1]);
                    t[c][e] = lo16(u);
                    t[c][e + 1] = hi16(u);
                }
            }
            ss += squares(t[c]);
        }
    }
    if (p.pre) {
        ss = sum_row<LANES>(ss, sums[1]);
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            unit(t[c], ss, p.d, p.eps);
            if (p.w_pre && col < p.d) {
                float w[8];
                load_w(p.w_pre, p.w_dtype, col, w);
#pragma unroll
                for (int e = 0; e < 8; e++) t[c][e] *= w[e];
            }
        }
    }
    if constexpr (QDQ != LA_QDQ_NONE) {
        float amax[CH];
#pragma unroll
        for (int c = 0; c < CH; c++) {
            amax[c] = 0.0f;
            if ((c * LANES + l) * kPiece < p.d) {
#pragma unroll
                for (int e = 0; e < 8; e++) amax[c] = larger_abs(amax[c], t[c][e]);
            }
        }
        emit_codes<QDQ, LANES, CH>(CodeOut{p.d, p.group, p.codes, p.scales}, l, row, base, t, amax, lds);
    }
    if (p.y) {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if (col < p.d) store8(static_cast<O*>(p.y) + base + col, t[c]);
        }
    }
}

// Backward, with r1 and r2 the reciprocal roots of the norms after and before a block:
//     T       = dh + r2 (dy w_pre - h r2^2 mean(dy w_pre h))   (pre)   or   dh + dy
//     dres    = T,   dalpha = sum T p,   G = alpha T
//     dz      = G n act'(z),   G <- G act(z)                     (gate last)
//     dw_post = sum G u r1,    G <- r1 (G w_post - u r1^2 mean(G w_post u))
//     dz      = G x act'(z),   G <- G act(z)                     (gate first)
//     dx      = G,             dw_pre = sum dy h r2.
// A workgroup walks rows a grid apart; the parameters' partial sums stay in registers (FP32, over its
// rows), are joined in double over the workgroup's rows in LDS and over workgroups by further kernels.
struct GateBwd {
    int rows, d, head, gate, first, post, pre, w_dtype;
    float eps;
    int64_t ld_x, ld_z;
    const void* x;
    const void* z;
    const void* w_post;
    const void* alpha;
    const void* h;
    const void* w_pre;
    const void* dy;
    const void* dh;
    void* dx;
    void* dz;
    void* dres;
    float* part[3];  // of w_post, alpha, w_pre: [workgroups][d], or null
};

template <class T, class O, int LANES, int CH>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void gate_bwd_kernel(GateBwd p) {
    constexpr int THREADS = LANES < 256 ? 256 : LANES, RPW = THREADS / LANES, WAVES = THREADS / 64;
    __shared__ float lds[2][3][WAVES];
    __shared__ float red[RPW > 1 ? THREADS * 8 : 1];
    const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    float sum[3][CH][8] = {};
    const float inv_d = 1.0f / static_cast<float>(p.d), inv_n = p.head ? 1.0f / static_cast<float>(p.head) : inv_d;
    const int head_lanes = p.head / kPiece;
    int par = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + sub; row < p.rows; row += static_cast<int64_t>(gridDim.x) * RPW) {
        const size_t base = static_cast<size_t>(row) * p.d;
        float x[CH][8] = {}, z[CH][8] = {}, h[CH][8] = {}, dy[CH][8] = {}, up[CH][8] = {};
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if (col < p.d) {
                load8(static_cast<const T*>(p.x) + row * p.ld_x + col, x[c]);
                if (p.z) load8(static_cast<const T*>(p.z) + row * p.ld_z + col, z[c]);
                if (p.pre) load8(static_cast<const T*>(p.h) + base + col, h[c]);
                load8(static_cast<const O*>(p.dy) + base + col, dy[c]);
                if (p.dh) load8(static_cast<const T*>(p.dh) + base + col, up[c]);
            }
        }
        float hh = 0.0f, gh = 0.0f, uu = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if (p.pre && col < p.d) {
                float w[8];
                load_w(p.w_pre, p.w_dtype, col, w);
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    hh = __builtin_fmaf(h[c][e], h[c][e], hh);
                    gh = __builtin_fmaf(dy[c][e] * w[e], h[c][e], gh);
                }
            }
            if (p.post && p.head == 0) {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float u = p.first ? x[c][e] * gate_of<T>(z[c][e], p.gate) : x[c][e];
                    uu = __builtin_fmaf(u, u, uu);
                }
            }
        }
        const bool whole = p.post && p.head == 0;
        if (p.pre || whole) {
            constexpr int N = LANES < 64 ? LANES : 64;
            if (p.pre) hh = sum_lanes(hh, N), gh = sum_lanes(gh, N);
            if (whole) uu = sum_lanes(uu, N);
            if constexpr (LANES > 64) {
                par ^= 1;
                if ((threadIdx.x & 63) == 0) {
                    lds[par][0][threadIdx.x >> 6] = hh;
                    lds[par][1][threadIdx.x >> 6] = gh;
                    lds[par][2][threadIdx.x >> 6] = uu;
                }
                __syncthreads();
                hh = gh = uu = 0.0f;
#pragma unroll
                for (int k = 0; k < WAVES; k++) {
                    hh += lds[par][0][k];
                    gh += lds[par][1][k];
                    uu += lds[par][2][k];
                }
            }
        }
        const float r2 = p.pre ? rsqrt_fine(hh * inv_d + p.eps) : 1.0f;
        const float k2 = gh * inv_d * r2 * r2;
        const float r_row = whole ? rsqrt_fine(uu * inv_n + p.eps) : 1.0f;
        // up: the gradient of n (post) or of u; x: u
        float gu = 0.0f, r1[CH], part[CH];
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            const bool in = col < p.d;
            float w[8], a[8], wp[8];
#pragma unroll
            for (int e = 0; e < 8; e++) w[e] = a[e] = wp[e] = 1.0f;
            if (in) {
                if (p.pre) load_w(p.w_pre, p.w_dtype, col, wp);
                if (p.alpha) load_w(p.alpha, p.w_dtype, col, a);
                if (p.post) load_w(p.w_post, p.w_dtype, p.head ? col & (p.head - 1) : col, w);
            }
            r1[c] = r_row;
            if (p.post && p.head) {
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float u = p.first ? x[c][e] * gate_of<T>(z[c][e], p.gate) : x[c][e];
                    s = __builtin_fmaf(u, u, s);
                }
                r1[c] = rsqrt_fine(sum_lanes(s, head_lanes) * inv_n + p.eps);
            }
            float dz[8];
            part[c] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float t = up[c][e];
                if (p.pre) {
                    t = __builtin_fmaf(r2, __builtin_fmaf(dy[c][e], wp[e], -h[c][e] * k2), t);
                    sum[2][c][e] = __builtin_fmaf(dy[c][e], h[c][e] * r2, sum[2][c][e]);
                } else {
                    t += dy[c][e];
                }
                float gate = 1.0f, slope = 0.0f;
                if (p.z) gate_both<T>(z[c][e], p.gate, gate, slope);
                const float u = p.first ? x[c][e] * gate : x[c][e];
                const float ur = u * r1[c], n = p.post ? ur * w[e] : u;
                const float out = p.first ? n : n * gate;  // p of the formula
                sum[1][c][e] = __builtin_fmaf(t, out, sum[1][c][e]);
                up[c][e] = t;
                float g = t * a[e];
                dz[e] = g * n * slope;
                if (!p.first) g *= gate;
                sum[0][c][e] = __builtin_fmaf(g, ur, sum[0][c][e]);
                dy[c][e] = p.post ? g * w[e] : g;  // (dy is used up: the gradient of u / rms)
                part[c] = __builtin_fmaf(dy[c][e], u, part[c]);
            }
            if (in && p.dres) store8(static_cast<T*>(p.dres) + base + col, up[c]);
            if (in && p.dz && !p.first) store8(static_cast<T*>(p.dz) + row * p.ld_z + col, dz);
            gu += part[c];
        }
        if (whole) {
            gu = sum_lanes(gu, LANES < 64 ? LANES : 64);
            if constexpr (LANES > 64) {
                par ^= 1;
                if ((threadIdx.x & 63) == 0) lds[par][0][threadIdx.x >> 6] = gu;
                __syncthreads();
                gu = 0.0f;
#pragma unroll
                for (int k = 0; k < WAVES; k++) gu += lds[par][0][k];
            }
        }
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            const float m = whole ? gu : p.post ? sum_lanes(part[c], head_lanes) : 0.0f;
            if (col >= p.d) continue;
            const float k1 = m * inv_n * r1[c] * r1[c];
            float dz[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float gate = 1.0f, slope = 0.0f;
                if (p.first) gate_both<T>(z[c][e], p.gate, gate, slope);
                float g = dy[c][e];
                if (p.post) g = r1[c] * __builtin_fmaf(-(p.first ? x[c][e] * gate : x[c][e]), k1, g);
                dz[e] = g * x[c][e] * slope;
                dy[c][e] = p.first ? g * gate : g;
            }
            if (p.dz && p.first) store8(static_cast<T*>(p.dz) + row * p.ld_z + col, dz);
            store8(static_cast<T*>(p.dx) + row * p.ld_x + col, dy[c]);
        }
    }
#pragma unroll
    for (int k = 0; k < 3; k++) {
        if (!p.part[k]) continue;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if constexpr (RPW > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; e++) red[threadIdx.x * 8 + e] = sum[k][c][e];
                __syncthreads();
                if (sub == 0) {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        double s = sum[k][c][e];
                        for (int i = 1; i < RPW; i++) s += red[(i * LANES + l) * 8 + e];
                        sum[k][c][e] = static_cast<float>(s);
                    }
                }
            }
            if (sub == 0 && col < p.d) store8(p.part[k] + static_cast<size_t>(blockIdx.x) * p.d + col, sum[k][c]);
        }
    }
}

// Lanes a row and pieces a lane, as in the residual norm.
template <class F>
hipError_t by_width(int d, F&& f) {
    using std::integral_constant;
    const int pieces = d / kPiece;
    if (pieces <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (pieces <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (pieces <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
    if (pieces <= 64) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (pieces <= 128) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (pieces <= 256) return f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (pieces <= 512) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    if (pieces <= 1024) return f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    return f(integral_constant<int, 256>{}, integral_constant<int, 8>{});
}
// The backward holds five rows: one piece a lane as long as a workgroup takes the row.
template <class F>
hipError_t by_width_bwd(int d, F&& f) {
    using std::integral_constant;
    const int pieces = d / kPiece;
    if (pieces <= 64) return by_width(d, f);
    if (pieces <= 256) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    if (pieces <= 512) return f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
    if (pieces <= 1024) return f(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
    return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}
template <class F>
hipError_t by_types(const la_gate_norm_config& c, F&& f) {
    if (c.x_dtype == LA_BF16) return c.out_dtype == LA_BF16 ? f(uint16_t{}, uint16_t{}) : f(uint16_t{}, float{});
    return c.out_dtype == LA_BF16 ? f(float{}, uint16_t{}) : f(float{}, float{});
}

int bwd_groups(const la_gate_norm_config& c) {
    const int pieces = c.d / kPiece, lanes = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : pieces <= 64 ? 64 : 256;
    const int rpw = 256 / lanes;
    const int need = (c.rows + rpw - 1) / rpw, most = c.d <= 1024 ? 2048 : c.d <= 4096 ? 1024 : 512;
    return need < most ? need : most;
}

}  // namespace

hipError_t launch_gate_fwd(const la_gate_norm_config& c, const GateArgs& a, hipStream_t s) {
    const GateFwd p{c.rows, c.d, c.head, c.gate, c.gate_first, c.post, c.pre, c.group, c.w_dtype, c.eps,
                    c.ld_x ? c.ld_x : c.d, c.ld_z ? c.ld_z : c.d, a.x, a.z, a.w_post, a.alpha, a.res, a.w_pre, a.h, a.y,
                    static_cast<uint8_t*>(a.codes), a.scales};
    return by_types(c, [&](auto t, auto o) {
        return by_width(c.d, [&](auto lanes, auto ch) {
            using T = decltype(t);
            using O = decltype(o);
            constexpr int LANES = decltype(lanes)::value, CH = decltype(ch)::value;
            const unsigned grid = static_cast<unsigned>((c.rows + 256 / LANES - 1) / (256 / LANES));
            switch (c.qdq) {
                case LA_QDQ_INT8_GROUP:
                    gate_fwd_kernel<T, O, LANES, CH, LA_QDQ_INT8_GROUP><<<grid, 256, 0, s>>>(p);
                    break;
                case LA_QDQ_E4M3_TILE:
                    gate_fwd_kernel<T, O, LANES, CH, LA_QDQ_E4M3_TILE><<<grid, 256, 0, s>>>(p);
                    break;
                default:
                    gate_fwd_kernel<T, O, LANES, CH, LA_QDQ_NONE><<<grid, 256, 0, s>>>(p);
            }
            return hipGetLastError();
        });
    });
}

size_t gate_bwd_workspace(const la_gate_norm_config& c) {
    return static_cast<size_t>(bwd_groups(c)) * c.d * sizeof(float) * 3;
}

hipError_t launch_gate_bwd(const la_gate_norm_config& c, const GateArgs& a, hipStream_t s) {
    const int groups = bwd_groups(c);
    const size_t one = static_cast<size_t>(groups) * c.d;
    float* const part[3] = {a.dw_post ? a.part : nullptr, a.dalpha ? a.part + one : nullptr, a.dw_pre ? a.part + 2 * one : nullptr};
    if (groups > 0) {
        const GateBwd p{c.rows, c.d, c.head, c.gate, c.gate_first, c.post, c.pre, c.w_dtype, c.eps,
                        c.ld_x ? c.ld_x : c.d, c.ld_z ? c.ld_z : c.d, a.x, a.z, a.w_post, a.alpha, a.h, a.w_pre, a.dy, a.dh,
                        a.dx, a.dz, a.dres, {part[0], part[1], part[2]}};
        const hipError_t e = by_types(c, [&](auto t, auto o) {
            return by_width_bwd(c.d, [&](auto lanes, auto ch) {
                constexpr int LANES = decltype(lanes)::value;
                gate_bwd_kernel<decltype(t), decltype(o), LANES, decltype(ch)::value><<<groups, LANES < 256 ? 256 : LANES, 0, s>>>(p);
                return hipGetLastError();
            });
        });
        if (e != hipSuccess) return e;
    }
    // a head's weight is shared by the row's heads: its sums run over them too
    const int wide = c.head ? c.head : c.d;
    if (a.dw_post)
        if (hipError_t e = launch_reduce_parts(part[0], groups * (c.d / wide), wide, a.dw_post, wide, nullptr, s)) return e;
    if (a.dalpha)
        if (hipError_t e = launch_reduce_parts(part[1], groups, c.d, a.dalpha, c.d, nullptr, s)) return e;
    if (a.dw_pre) return launch_reduce_parts(part[2], groups, c.d, a.dw_pre, c.d, nullptr, s);
    return hipSuccess;
}

}  // namespace la
