// RMS norm of the residual stream: h = rne(x + residual), n = h rstd w, with an optional 8-bit
// codec on n, and its backward.
//
// One pass over the data: a row's values stay in registers between the sum of squares and the
// output, so x and residual are read once and each output written once; memory bound.  A row
// is held by LANES lanes (8 to 64 of one wave, or 256 = a workgroup's four waves), each lane
// CH pieces of 8 consecutive columns, the pieces of neighbouring lanes next to each other: 16
// or 32 bytes a lane and access, and a codec's group of 16..128 columns is 2..16 neighbouring
// lanes, whose maximum needs no LDS.  bf16: 40686 rows of 4096 to INT8 codes with a scale for 64
// and their values 270 us by the clock, 283 by the profiler (5.3 TB/s, the vector units 73% busy);
// 32768 rows of 2048 forward 100 us (5.4 TB/s), backward 114 us (4.8 TB/s) and 5 us for the weight's
// sums; 256 rows of 2048 to E4M3 7.8 us, latencies (64 of the chip's 256 CUs have rows).
#include "la_layer.hpp"

namespace la {
namespace {

constexpr int kPiece = 8;

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        widen(load16(p), v);
    } else {
        float a[4], b[4];
        widen(load16(p), a);
        widen(load16(p + 4), b);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        store16(p, narrow(v));
    } else {
        store16(p, uv4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
        store16(p + 4, uv4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
    }
}
__device__ __forceinline__ void load_w(const void* w, int dtype, int col, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = 1.0f;
    } else if (dtype == LA_BF16) {
        load8(static_cast<const uint16_t*>(w) + col, v);
    } else {
        load8(static_cast<const float*>(w) + col, v);
    }
}

// The larger of a magnitude and |b|, a NaN above every number (fmaxf would drop it).
__device__ __forceinline__ float larger_abs(float a, float b) {
    const uint32_t u = __float_as_uint(a), v = __float_as_uint(b) & 0x7FFFFFFFu;
    return __uint_as_float(u > v ? u : v);
}

// Sum over the row's lanes, the same bits in each of them.
template <int LANES>
__device__ __forceinline__ float row_sum(float x, float* lds) {
    if constexpr (LANES <= 64) return group_sum<LANES>(x);
    x = group_sum<64>(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}
// Two sums at once, by one barrier: `lds` is another eight words in the next call.
template <int LANES>
__device__ __forceinline__ void row_sums(float& a, float& b, float* lds) {
    a = group_sum<(LANES < 64 ? LANES : 64)>(a);
    b = group_sum<(LANES < 64 ? LANES : 64)>(b);
    if constexpr (LANES <= 64) return;
    if ((threadIdx.x & 63) == 0) {
        lds[threadIdx.x >> 6] = a;
        lds[4 + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    b = (lds[4] + lds[5]) + (lds[6] + lds[7]);
}
__device__ __forceinline__ double join64(uint32_t lo, uint32_t hi) {
    return __builtin_bit_cast(double, static_cast<uint64_t>(lo) | (static_cast<uint64_t>(hi) << 32));
}
template <int CTRL>
__device__ __forceinline__ double dpp_double(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return join64(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xF, 0xF, true),
                  __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xF, 0xF, true));
}
// The sum of doubles, by the exchanges of group_sum (by shuffles: 14.2 us against 12.7 for 40000 rows of 128).
template <int LANES>
__device__ __forceinline__ double row_sum_wide(double x, double* lds) {
    if (LANES >= 2) x += dpp_double<kDppXor1>(x);
    if (LANES >= 4) x += dpp_double<kDppXor2>(x);
    if (LANES >= 8) x += dpp_double<kDppHalfMirror>(x);
    if (LANES >= 16) x += dpp_double<kDppMirror>(x);
    if (LANES >= 32) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint32_t a = static_cast<uint32_t>(u), b = static_cast<uint32_t>(u >> 32);
        const auto lo = __builtin_amdgcn_permlane16_swap(a, a, false, false), hi = __builtin_amdgcn_permlane16_swap(b, b, false, false);
        x = join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
    }
    if (LANES >= 64) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint32_t a = static_cast<uint32_t>(u), b = static_cast<uint32_t>(u >> 32);
        const auto lo = __builtin_amdgcn_permlane32_swap(a, a, false, false), hi = __builtin_amdgcn_permlane32_swap(b, b, false, false);
        x = join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
    }
    if constexpr (LANES <= 64) return x;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}
template <int LANES>
__device__ __forceinline__ float row_max(float x, float* lds) {
    if constexpr (LANES <= 64) return group_max_abs<LANES>(x);
    x = group_max_abs<64>(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[4 + (threadIdx.x >> 6)] = x;
    __syncthreads();
    return larger_abs(larger_abs(lds[4], lds[5]), larger_abs(lds[6], lds[7]));
}

// 1 / sqrt(m), correct to about an ulp: the hardware's estimate and one Newton step (skipped
// where the estimate is 0, infinite or NaN).
__device__ __forceinline__ float rsqrt_fine(float m) {
    const float r = __builtin_amdgcn_rsqf(m);
    const float e = __builtin_fmaf(-m * r, r, 1.0f);
    const float y = __builtin_fmaf(0.5f * r, e, r);
    return (m > 1e-35f && m < 1e35f) ? y : 1.0f / sqrtf(m);
}

struct NormFwd {
    int rows, d, w_dtype, group;
    float eps;
    const void* x;
    const void* res;
    const void* w;
    void* res_out;
    void* y;
    uint8_t* codes;
    float* scales;
};

template <class T, class O, int LANES, int CH, int QDQ>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormFwd p) {
    constexpr int RPW = 256 / LANES;  // rows a workgroup
    // Codes: every operation is rounded as the formula has it (the squares summed in double), and a
    // value near the middle between two codes goes where FP32 arithmetic puts it, whatever y's type
    // and whether y is wanted at all.
    constexpr bool STEPWISE = QDQ != LA_QDQ_NONE;
    __shared__ float lds[8];
    __shared__ double wide[STEPWISE ? 4 : 1];
    const int l = threadIdx.x % LANES;
    const int row = blockIdx.x * RPW + threadIdx.x / LANES;
    if (LANES <= 64 && row >= p.rows) return;  // whole groups of lanes leave together
    const size_t base = static_cast<size_t>(row) * p.d;
    float h[CH][8];
    std::conditional_t<STEPWISE, double, float> ss = 0;
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int col = (c * LANES + l) * kPiece;
        if (col < p.d) {
            load8(static_cast<const T*>(p.x) + base + col, h[c]);
            if (p.res) {
                float r[8];
                load8(static_cast<const T*>(p.res) + base + col, r);
#pragma unroll
                for (int e = 0; e < 8; e++) h[c][e] += r[e];
            }
            if constexpr (sizeof(T) == 2) {  // the norm reads what res_out holds
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const uint32_t u = pack16(h[c][e], h[c][e + 1]);
                    h[c][e] = lo16(u);
                    h[c][e + 1] = hi16(u);
                }
            }
            if (p.res_out) store8(static_cast<T*>(p.res_out) + base + col, h[c]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) h[c][e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if constexpr (STEPWISE) ss += h[c][e] * h[c][e];
            else ss = __builtin_fmaf(h[c][e], h[c][e], ss);
        }
    }
    float r;  // 1 / rms, or the rms
    [[maybe_unused]] float recip = 0.0f;  // RN(1 / r) as in int8_scale_recip, where its quotients are the exact ones
    [[maybe_unused]] bool by_recip = false;
    if constexpr (STEPWISE) {
        r = sqrtf(static_cast<float>(row_sum_wide<LANES>(ss, wide) / p.d) + p.eps);
        by_recip = r > 0x1p-60f && r < 0x1p60f;
        const float e = __builtin_amdgcn_rcpf(r);
        recip = __builtin_fmaf(__builtin_fmaf(-r, e, 1.0f), e, e);
    } else {
        r = rsqrt_fine(row_sum<LANES>(ss, lds) / static_cast<float>(p.d) + p.eps);
    }
    float amax[CH];
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int col = (c * LANES + l) * kPiece;
        float w[8];
        amax[c] = 0.0f;
        if (col < p.d) {
            load_w(p.w, p.w_dtype, col, w);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                if constexpr (STEPWISE) h[c][e] = (by_recip ? quot_rn_fast(h[c][e], r, recip) : h[c][e] / r) * w[e];
                else h[c][e] = h[c][e] * r * w[e];
                if (QDQ != LA_QDQ_NONE) amax[c] = larger_abs(amax[c], h[c][e]);
            }
        }
    }
    if constexpr (QDQ != LA_QDQ_NONE) {
        if (p.group == 0) {
            float m = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; c++) m = larger_abs(m, amax[c]);
            m = row_max<LANES>(m, lds);
#pragma unroll
            for (int c = 0; c < CH; c++) amax[c] = m;
        } else {  // a row of LANES * 8 columns or more holds whole groups; in a shorter one a group may be the row
#pragma unroll
            for (int c = 0; c < CH; c++) {
                amax[c] = group_max_abs<2>(amax[c]);
                if (p.group >= 32) amax[c] = larger_abs(amax[c], dpp<kDppXor2>(amax[c]));
                if (p.group >= 64) amax[c] = larger_abs(amax[c], dpp<kDppHalfMirror>(amax[c]));
                if (p.group >= 128) amax[c] = larger_abs(amax[c], dpp<kDppMirror>(amax[c]));
            }
        }
        const int per_row = p.group ? p.d / p.group : 1;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if (col >= p.d) continue;
            float s, y;
            uint32_t word[2] = {0, 0};
            // a NaN in the group: its maximum, its scale and every value that its codes stand for
            const bool none = amax[c] != amax[c];
            if constexpr (QDQ == LA_QDQ_INT8_GROUP) {
                bool fast = int8_scale_recip(amax[c], s, y);
                if (none) s = amax[c], fast = false;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    float q = fast ? int8_code_fast(h[c][e], s, y) : rintf(h[c][e] / s);
                    const bool number = q == q;  // (of a quotient without one: code 0)
                    if (!fast && number) q = fminf(fmaxf(q, -127.0f), 127.0f);
                    word[e >> 2] |= (number ? static_cast<uint32_t>(static_cast<int>(q)) & 0xFFu : 0u) << (8 * (e & 3));
                    h[c][e] = q * s;
                }
            } else {
                bool fast = e4m3_scale_recip(amax[c], s, y);
                if (none) s = amax[c], fast = false;
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float a = fast ? quot_rn_fast(h[c][e], s, y) : h[c][e] / s;
                    float b = fast ? quot_rn_fast(h[c][e + 1], s, y) : h[c][e + 1] / s;
                    a = a != a ? a : fminf(fmaxf(a, -448.0f), 448.0f);
                    b = b != b ? b : fminf(fmaxf(b, -448.0f), 448.0f);
                    const uint32_t k = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false)) & 0xFFFFu;
                    word[e >> 2] |= k << (8 * (e & 3));
                    h[c][e] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(k), 0) * s;
                    h[c][e + 1] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(k), 1) * s;
                }
            }
            if (p.codes) *reinterpret_cast<uv2*>(p.codes + base + col) = uv2{word[0], word[1]};
            if (p.scales) {
                if (p.group ? col % p.group == 0 : col == 0)
                    p.scales[static_cast<size_t>(row) * per_row + (p.group ? col / p.group : 0)] = s;
            }
        }
    }
    if (p.y) {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if (col < p.d) store8(static_cast<O*>(p.y) + base + col, h[c]);
        }
    }
}

// Backward: with r = rstd and g = dy w,  dx = dres + r (g - h r^2 mean(g h)),  dw = sum dy h r.
// A workgroup walks rows a grid apart, dw's partial sums in registers (FP32); they are joined in
// double over the workgroup's rows in LDS and over workgroups by a second kernel, in a fixed order.
struct NormBwd {
    int rows, d, w_dtype;
    float eps;
    const void* h;
    const void* w;
    const void* dy;
    const void* dres;
    void* dx;
    float* part;  // [workgroups][d], or null
};

template <class T, class O, int LANES, int CH>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormBwd p) {
    constexpr int RPW = 256 / LANES;
    __shared__ float lds[2][8];
    __shared__ float red[LANES <= 64 ? 256 * 8 : 1];
    const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    float dw[CH][8] = {};
    int par = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + sub; row < p.rows; row += static_cast<int64_t>(gridDim.x) * RPW) {
        const size_t base = static_cast<size_t>(row) * p.d;
        float h[CH][8], dy[CH][8], up[CH][8] = {};
        float ss = 0.0f, gh = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            float w[8];
            if (col < p.d) {
                load8(static_cast<const T*>(p.h) + base + col, h[c]);
                load8(static_cast<const O*>(p.dy) + base + col, dy[c]);
                load_w(p.w, p.w_dtype, col, w);
                if (p.dres) load8(static_cast<const T*>(p.dres) + base + col, up[c]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) h[c][e] = dy[c][e] = w[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; e++) {
                ss = __builtin_fmaf(h[c][e], h[c][e], ss);
                gh = __builtin_fmaf(dy[c][e] * w[e], h[c][e], gh);
            }
        }
        const float inv = 1.0f / static_cast<float>(p.d);
        row_sums<LANES>(ss, gh, lds[par ^= 1]);
        const float r = rsqrt_fine(ss / static_cast<float>(p.d) + p.eps);
        const float k = gh * inv * r * r;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if (col >= p.d) continue;
            float w[8];
            load_w(p.w, p.w_dtype, col, w);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float hr = h[c][e] * r;
                dw[c][e] = __builtin_fmaf(dy[c][e], hr, dw[c][e]);
                up[c][e] = __builtin_fmaf(r, __builtin_fmaf(dy[c][e], w[e], -h[c][e] * k), up[c][e]);
            }
            store8(static_cast<T*>(p.dx) + base + col, up[c]);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int col = (c * LANES + l) * kPiece;
        if constexpr (RPW > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; e++) red[threadIdx.x * 8 + e] = dw[c][e];
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    double s = dw[c][e];
                    for (int k = 1; k < RPW; k++) s += red[(k * LANES + l) * 8 + e];
                    dw[c][e] = static_cast<float>(s);
                }
            }
        }
        if (sub == 0 && col < p.d) store8(p.part + static_cast<size_t>(blockIdx.x) * p.d + col, dw[c]);
    }
}

// Lanes a row and pieces a lane: the fewest lanes that hold the row in one piece each up to a
// wave, then up to four pieces a lane in one wave (2048 columns: no LDS in the sums), then a
// workgroup.
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
// The backward holds three rows: one piece a lane as long as a workgroup takes the row.
template <class F>
hipError_t by_width_bwd(int d, F&& f) {
    using std::integral_constant;
    const int pieces = d / kPiece;
    if (pieces > 64 && pieces <= 256) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    return by_width(d, f);
}
template <class F>
hipError_t by_types(const la_norm_config& c, F&& f) {
    if (c.x_dtype == LA_BF16) return c.out_dtype == LA_BF16 ? f(uint16_t{}, uint16_t{}) : f(uint16_t{}, float{});
    return c.out_dtype == LA_BF16 ? f(float{}, uint16_t{}) : f(float{}, float{});
}

int norm_lanes(int d) {
    const int pieces = d / kPiece;
    return pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : pieces <= 64 ? 64 : 256;
}
// Workgroups of the backward: as many as the chip holds (by the pieces a lane holds of three
// rows: 8, 4 or 2 a CU), half of that where the partial sums, read again, outweigh it
// (d = 2048: 218 us for 32768 rows forward and backward with 1024, 223 with 2048, 240 with 512;
// d = 1024, 65536 rows: 209 with 2048, 230 with 1024).
int norm_bwd_groups(const la_norm_config& c) {
    const int rpw = 256 / norm_lanes(c.d);
    const int need = (c.rows + rpw - 1) / rpw, most = c.d <= 1024 ? 2048 : c.d <= 4096 ? 1024 : 512;
    return need < most ? need : most;
}

}  // namespace

hipError_t launch_norm_fwd(const la_norm_config& c, const NormArgs& a, hipStream_t s) {
    const NormFwd p{c.rows, c.d, c.w_dtype, c.group, c.eps, a.x, a.res, a.w, a.res_out, a.y,
                    static_cast<uint8_t*>(a.codes), a.scales};
    return by_types(c, [&](auto t, auto o) {
        return by_width(c.d, [&](auto lanes, auto ch) {
            using T = decltype(t);
            using O = decltype(o);
            constexpr int LANES = decltype(lanes)::value, CH = decltype(ch)::value;
            const unsigned grid = static_cast<unsigned>((c.rows + 256 / LANES - 1) / (256 / LANES));
            switch (c.qdq) {
                case LA_QDQ_INT8_GROUP:
                    norm_fwd_kernel<T, O, LANES, CH, LA_QDQ_INT8_GROUP><<<grid, 256, 0, s>>>(p);
                    break;
                case LA_QDQ_E4M3_TILE:
                    norm_fwd_kernel<T, O, LANES, CH, LA_QDQ_E4M3_TILE><<<grid, 256, 0, s>>>(p);
                    break;
                default:
                    norm_fwd_kernel<T, O, LANES, CH, LA_QDQ_NONE><<<grid, 256, 0, s>>>(p);
            }
            return hipGetLastError();
        });
    });
}

size_t norm_bwd_workspace(const la_norm_config& c) {
    return static_cast<size_t>(norm_bwd_groups(c)) * c.d * sizeof(float);
}

hipError_t launch_norm_bwd(const la_norm_config& c, const NormArgs& a, hipStream_t s) {
    const int groups = norm_bwd_groups(c);
    if (groups > 0) {
        const NormBwd p{c.rows, c.d, c.w_dtype, c.eps, a.x, a.w, a.dy, a.dres, a.dx, a.dw ? a.part : nullptr};
        const hipError_t e = by_types(c, [&](auto t, auto o) {
            return by_width_bwd(c.d, [&](auto lanes, auto ch) {
                norm_bwd_kernel<decltype(t), decltype(o), decltype(lanes)::value, decltype(ch)::value>
                    <<<groups, 256, 0, s>>>(p);
                return hipGetLastError();
            });
        });
        if (e != hipSuccess) return e;
    }
    if (!a.dw) return hipSuccess;
    return launch_reduce_parts(a.part, groups, c.d, a.dw, c.d, nullptr, s);
}

}  // namespace la
