// Norms around a block with its gate and residual scale:
//     u = x act(z) (gate first) or x,   n = u / rms(u over a head or the row) * w_post,
//     p = n act(z) (gate last) or n,    t = residual + alpha p,   h = rne(t),
//     v = h / rms(h) * w_pre  or t,     and 8-bit codes of v,
// Memory bound: one pass over the data, a row in the registers of 8 to 384 lanes between its loads, its
// two norms and its outputs.  A head of 16 to 512 columns is 2 to 64 neighbouring lanes, whose sum needs no
// LDS.  bf16 to INT8 codes and their values: 40686 rows of 32 heads of 128 with silu 206 us (5.6 TB/s), the join of
// 40686 x 2048 154 us (4.9 TB/s): by the vector units as much as by memory; 32768 x 2048 without codes 70 and 108 us; 4 rows
// of 2048 3.5 us, latencies.  E4M3 as INT8 (213 and 153); FP32 rows to INT8, every operation as the formula has it,
// 20343 rows 190 and 134 us (5.7 and 5.3 TB/s), codes alone of 8192 x 2048 without norms 14.
#include "la_gate.hpp"

namespace la {
namespace {

// The gate as its formula is rounded, operation by operation.
__device__ __forceinline__ float gate_stepwise(float z, int gate) {
    const float s = 1.0f / (1.0f + expf(-z));
    return gate == LA_GATE_SILU ? (z < -89.0f ? 0.0f : z * s) : s;
}

struct GateFwd {
    int rows, d, head, gate, first, post, pre, group, w_dtype, out_dtype;
    float eps;
    double inv_d, inv_head;
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

__device__ __forceinline__ void store_as(void* p, int dtype, size_t at, const float (&v)[8]) {
    if (dtype == LA_BF16) store8(static_cast<uint16_t*>(p) + at, v);
    else store8(static_cast<float*>(p) + at, v);
}

template <class T, int LANES, int CH, int QDQ, bool FINE>
__global__ __launch_bounds__(LANES <= 64 ? 256 : LANES) void gate_fwd_kernel(GateFwd p) {
    constexpr int RPW = LANES <= 64 ? 256 / LANES : 1;
    // What codes are formed from does not depend on y's type or on whether y is wanted.  Of FP32 rows every
    // operation is rounded as the formula has it and squares are summed in double, as in the residual norm
    // (STEPWISE); of bf16 rows (whose own rounding is 2^-8) sums are FP32, norms by the reciprocal root and the gate
    // within (|z| + 2) 2^-23 (40686 x 4096 with 32 heads of 128 and silu: 289 us stepwise, 206 so).  Codes are those of
    // the correctly rounded quotient in both (by the product with the scale's reciprocal, which may take a near tie
    // to the other side, bf16 rows took 200 us, and the join of 40686 x 2048 150 for 154).  Where h is
    // rounded before the next norm, what leads to it is rounded stepwise too and a row's sum joined in double
    // (FINE), with codes and without: a last bit there moves h by 2^-8 of itself where it falls on a tie, and with a
    // row's largest element its scale (40686 x 2048: 530 of 83 million elements differ from the formula so rounded
    // without it and 170, by the mean's last bit, with it; it takes about 1 us).
    constexpr bool STEPWISE = QDQ != LA_QDQ_NONE && sizeof(T) == 4;
    typedef std::conditional_t<FINE, double, float> S;
    typedef std::conditional_t<STEPWISE, double, float> S2;
    __shared__ S sums[LANES / 64 + 1];
    __shared__ S2 sums2[LANES / 64 + 1];
    __shared__ float lds[LANES / 64 + 1];
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
            for (int e = 0; e < 8; e++) {
                if constexpr (FINE) g[c][e] = gate_stepwise(g[c][e], p.gate);
                else g[c][e] = gate_of<T>(g[c][e], p.gate);
            }
        if (p.first) {
#pragma unroll
            for (int c = 0; c < CH; c++)
#pragma unroll
                for (int e = 0; e < 8; e++) t[c][e] *= g[c][e];
        }
    }
    const float inv_d = 1.0f / static_cast<float>(p.d), inv_head = 1.0f / static_cast<float>(p.head ? p.head : 1);
    // v / rms: stepwise by the correctly rounded quotient, else by the reciprocal root
    auto unit = [&p](auto fine, float (&v)[8], auto sum, int n, [[maybe_unused]] float inv, float eps) {
        if constexpr (decltype(fine)::value) {
            // (a double's quotient took 3 us of 152 here; its reciprocal's product rounds to the same FP32 value but
            // within 2^-52 of a tie)
            const float rms = sqrtf(static_cast<float>(sum * (n == p.d ? p.inv_d : p.inv_head)) + eps);
            const bool fast = rms > 0x1p-60f && rms < 0x1p60f;
            const float e0 = __builtin_amdgcn_rcpf(rms);
            const float recip = __builtin_fmaf(__builtin_fmaf(-rms, e0, 1.0f), e0, e0);
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = fast ? quot_rn_fast(v[e], rms, recip) : v[e] / rms;
        } else {
            const float k = rsqrt_fine(sum * inv + eps);
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] *= k;
        }
    };
    auto squares = [](auto zero, const float (&v)[8]) {
        auto s = zero;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if constexpr (sizeof(s) == 8) s += v[e] * v[e];
            else s = __builtin_fmaf(v[e], v[e], s);
        }
        return s;
    };
    if (p.post) {
        S row_ss = 0;
        if (p.head == 0) {
#pragma unroll
            for (int c = 0; c < CH; c++) row_ss += squares(S2(0), t[c]);
            row_ss = sum_row<LANES>(row_ss, sums);
        }
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            const S ss = p.head ? sum_lanes(squares(S(0), t[c]), p.head / kPiece) : row_ss;
            unit(std::bool_constant<FINE>{}, t[c], ss, p.head ? p.head : p.d, p.head ? inv_head : inv_d, p.eps);
            float w[8];
            if (p.w_post && col < p.d) {
                load_w(p.w_post, p.w_dtype, p.head ? col & (p.head - 1) : col, w);
#pragma unroll
                for (int e = 0; e < 8; e++) t[c][e] *= w[e];
            }
        }
    }
    S2 ss = 0;
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
            ss += squares(S2(0), t[c]);
        }
    }
    if (p.pre) {
        ss = sum_row<LANES>(ss, sums2);
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            unit(std::bool_constant<STEPWISE>{}, t[c], ss, p.d, inv_d, p.eps);
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
        const CodeOut o{p.d, p.group, p.codes, p.scales};
        emit_codes<QDQ, LANES, CH>(o, l, row, base, t, amax, lds);
    }
    if (p.y) {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if (col < p.d) store_as(p.y, p.out_dtype, base + col, t[c]);
        }
    }
}

// Lanes a row (gate_lanes) and pieces a lane: one piece a lane as far as that goes (a wave with up to four
// pieces a lane, as in the residual norm, took 189 us where a workgroup a row takes 149, of 40686 x 2048
// joined and to INT8), two of 256 lanes and more from there on.
template <class F>
hipError_t by_width(int d, F&& f) {
    using std::integral_constant;
    constexpr integral_constant<int, 1> one;
    switch (gate_lanes(d)) {
        case 8: return f(integral_constant<int, 8>{}, one);
        case 16: return f(integral_constant<int, 16>{}, one);
        case 32: return f(integral_constant<int, 32>{}, one);
        case 64: return f(integral_constant<int, 64>{}, one);
        case 128: return f(integral_constant<int, 128>{}, one);
        case 192: return f(integral_constant<int, 192>{}, one);
        case 384: return f(integral_constant<int, 384>{}, one);
    }
    const int pieces = d / kPiece;
    if (pieces <= 256) return f(integral_constant<int, 256>{}, one);
    if (pieces <= 512) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    if (pieces <= 1024) return f(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    return f(integral_constant<int, 256>{}, integral_constant<int, 8>{});
}
template <class F>
hipError_t by_type(const la_gate_norm_config& c, F&& f) {
    return c.x_dtype == LA_BF16 ? f(uint16_t{}) : f(float{});
}

}  // namespace

hipError_t launch_gate_fwd(const la_gate_norm_config& c, const GateArgs& a, hipStream_t s) {
    const GateFwd p{c.rows, c.d, c.head, c.gate, c.gate_first, c.post, c.pre, c.group, c.w_dtype, c.out_dtype, c.eps, 1.0 / c.d, 1.0 / (c.head ? c.head : 1),
                    c.ld_x ? c.ld_x : c.d, c.ld_z ? c.ld_z : c.d, a.x, a.z, a.w_post, a.alpha, a.res, a.w_pre, a.h, a.y,
                    static_cast<uint8_t*>(a.codes), a.scales};
    return by_type(c, [&](auto t) {
        return by_width(c.d, [&](auto lanes, auto ch) {
            using T = decltype(t);
            constexpr int LANES = decltype(lanes)::value, CH = decltype(ch)::value;
            constexpr int threads = LANES <= 64 ? 256 : LANES, rows = threads / LANES;
            const unsigned grid = static_cast<unsigned>((c.rows + rows - 1) / rows);
            auto launch = [&](auto qdq, auto fine) { gate_fwd_kernel<T, LANES, CH, decltype(qdq)::value, decltype(fine)::value><<<grid, threads, 0, s>>>(p); };
            // (h of FP32 rows is not rounded: there only codes ask for every operation as the formula has it)
            const bool rounded = sizeof(T) == 2 && c.pre && (c.post || c.gate);
            auto coded = [&](auto qdq) {
                if constexpr (sizeof(T) == 4) launch(qdq, std::bool_constant<decltype(qdq)::value != LA_QDQ_NONE>{});
                else if (rounded) launch(qdq, std::true_type{});
                else launch(qdq, std::false_type{});
            };
            switch (c.qdq) {
                case LA_QDQ_INT8_GROUP: coded(std::integral_constant<int, LA_QDQ_INT8_GROUP>{}); break;
                case LA_QDQ_E4M3_TILE: coded(std::integral_constant<int, LA_QDQ_E4M3_TILE>{}); break;
                default: coded(std::integral_constant<int, LA_QDQ_NONE>{});
            }
            return hipGetLastError();
        });
    });
}

}  // namespace la
