// Gradients of the norms around a block with its gate and residual scale.
//
// With r1 and r2 the reciprocal roots of the norms after and before a block:
//     T       = dh + r2 (dy w_pre - h r2^2 mean(dy w_pre h))   (pre)   or   dh + dy
//     dres    = T,   dalpha = sum T p,   G = alpha T
//     dz      = G n act'(z),   G <- G act(z)                     (gate last)
//     dw_post = sum G u r1,    G <- r1 (G w_post - u r1^2 mean(G w_post u))
//     dz      = G x act'(z),   G <- G act(z)                     (gate first)
//     dx      = G,             dw_pre = sum dy h r2.
// A workgroup walks up to 128 rows a grid apart; the parameters' partial sums stay in registers (FP32, over its
// rows), are joined in double over the workgroup's groups of lanes in LDS and over workgroups by a second kernel.
#include "la_gate.hpp"

namespace la {
namespace {

struct GateBwd {
    int rows, d, head, gate, post, w_dtype, out_dtype;
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
    float* part[3];  // of w_post ([workgroups][head or d]), alpha and w_pre ([workgroups][d]), or null
};

// A lane's piece of a row as it lies in memory: eight values of bf16 or of float.
struct Raw {
    uv4 a, b;
};
__device__ __forceinline__ Raw fetch_raw(const void* p, int dtype, size_t at) {
    Raw r{};
    if (dtype == LA_BF16) {
        r.a = load16(static_cast<const uint16_t*>(p) + at);
    } else {
        r.a = load16(static_cast<const float*>(p) + at);
        r.b = load16(static_cast<const float*>(p) + at + 4);
    }
    return r;
}
__device__ __forceinline__ void widen_raw(const Raw& r, int dtype, float (&v)[8]) {
    if (dtype == LA_BF16) {
        widen(r.a, v);
    } else {
        float a[4], b[4];
        widen(r.a, a);
        widen(r.b, b);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    }
}

enum GateAt { kNoGate, kGateLast, kGateFirst };

// Waves a SIMD that a kernel's registers leave room for, and workgroups a CU by them: all that a launch has are
// resident.  32768 x 2048 bf16, forward and backward: three 291 us (row norms) and 228 (head norms and
// gate), two 318 and 243, four, which spill, 426 and 296; gate and both norms: two 332 us, three, which
// spill, 452.  Some spill all the same: gate and both norms of up to 64 columns (80 registers, with 32 groups of
// lanes to join) and of 4097 to 8192 (6 with the gate last, 46 to 49 first); beyond 8192 columns all do (42 to 224).
constexpr int waves_for(int lanes, bool full) { return lanes <= 384 ? (full ? 2 : 3) : lanes == 512 ? 2 : 4; }  // full: gate and both norms
constexpr int groups_for(int lanes, bool full) { return lanes <= 64 ? waves_for(lanes, full) : 4 * waves_for(lanes, full) / (lanes / 64); }

// The loads of a workgroup's next row run under the sums of the one before: a row is five loads wide and
// two barriers long.  32768 x 2048 bf16: row norms and residual 160 us (5.1 TB/s), head norms and gate 130 us
// (5.1 TB/s): memory bound.  Wide rows, both norms without a gate, with all they write: 8192 rows of 6144 171 us
// and of 8192 190, 4096 rows of 16384 680.
template <class T, int LANES, int CH, GateAt GATE, bool PRE>
__global__ __launch_bounds__(LANES <= 64 ? 256 : LANES, waves_for(LANES, GATE != kNoGate && PRE)) void gate_bwd_kernel(GateBwd p) {
    constexpr int THREADS = LANES <= 64 ? 256 : LANES, RPW = THREADS / LANES, WAVES = THREADS / 64, CODE = Io<T>::kCode;
    constexpr bool AHEAD = CH == 1;  // (registers: two pieces a lane leave no room for a second row and the weights)
    __shared__ float lds[2][3][WAVES];
    __shared__ float red[THREADS * 8 * CH];
    const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    float sum[3][CH][8] = {};
    const float inv_d = 1.0f / static_cast<float>(p.d), inv_n = p.head ? 1.0f / static_cast<float>(p.head) : inv_d;
    const int head_lanes = p.head / kPiece;
    const bool whole = p.post && p.head == 0;
    int par = 0;
    // the weights of a piece: kept where registers allow it, else read again
    enum { kPost, kAlpha, kPre };
    float kept[3][AHEAD ? CH : 1][8];
    auto read_weight = [&](int which, int c, float (&w)[8]) {
        const int col = (c * LANES + l) * kPiece;
        const void* from = which == kPost ? p.w_post : which == kAlpha ? p.alpha : p.w_pre;
#pragma unroll
        for (int e = 0; e < 8; e++) w[e] = 1.0f;
        if (from && col < p.d) load_w(from, p.w_dtype, which == kPost && p.head ? col & (p.head - 1) : col, w);
    };
    auto weight = [&](int which, int c, float (&w)[8]) {
        if constexpr (AHEAD) {
#pragma unroll
            for (int e = 0; e < 8; e++) w[e] = kept[which][c][e];
        } else {
            read_weight(which, c, w);
        }
    };
    if constexpr (AHEAD) {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            read_weight(kPost, c, kept[kPost][c]);
            read_weight(kAlpha, c, kept[kAlpha][c]);
            if constexpr (PRE) read_weight(kPre, c, kept[kPre][c]);
        }
    }
    struct Row {
        Raw x, z, h, dy, dh;
    } next[CH];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            next[c] = Row{};
            if (row < p.rows && col < p.d) {
                const size_t at = static_cast<size_t>(row) * p.d + col;
                next[c].x = fetch_raw(p.x, CODE, row * p.ld_x + col);
                if (GATE != kNoGate) next[c].z = fetch_raw(p.z, CODE, row * p.ld_z + col);
                if (PRE) next[c].h = fetch_raw(p.h, CODE, at);
                next[c].dy = fetch_raw(p.dy, p.out_dtype, at);
                if (p.dh) next[c].dh = fetch_raw(p.dh, CODE, at);
            }
        }
    };
    const int64_t stride = static_cast<int64_t>(gridDim.x) * RPW;
    int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + sub;
    if constexpr (AHEAD) fetch(row);
    for (; row < p.rows; row += stride) {
        const size_t base = static_cast<size_t>(row) * p.d;
        if constexpr (!AHEAD) fetch(row);
        float x[CH][8], z[CH][8], h[CH][8], dy[CH][8], up[CH][8], gates[2][AHEAD ? CH : 1][8];
#pragma unroll
        for (int c = 0; c < CH; c++) {
            widen_raw(next[c].x, CODE, x[c]);
            if constexpr (GATE != kNoGate) widen_raw(next[c].z, CODE, z[c]);
            if constexpr (PRE) widen_raw(next[c].h, CODE, h[c]);
            widen_raw(next[c].dy, p.out_dtype, dy[c]);
            widen_raw(next[c].dh, CODE, up[c]);
        }
        if constexpr (AHEAD) fetch(row + stride);
        // the gate and its slope: kept, or formed again, as the weights
        [[maybe_unused]] auto gate_at = [&](int c, int e, float& gate, float& slope) {
            if constexpr (AHEAD) gate = gates[0][c][e], slope = gates[1][c][e];
            else gate_both<T>(z[c][e], p.gate, gate, slope);
        };
        float hh = 0.0f, gh = 0.0f, uu = 0.0f, us[CH];
#pragma unroll
        for (int c = 0; c < CH; c++) {
            us[c] = 0.0f;
            float w_pre[8];
            if constexpr (PRE) weight(kPre, c, w_pre);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                [[maybe_unused]] float gate, slope;
                if constexpr (GATE != kNoGate && (AHEAD || GATE == kGateFirst)) gate_both<T>(z[c][e], p.gate, gate, slope);
                if constexpr (GATE != kNoGate && AHEAD) gates[0][c][e] = gate, gates[1][c][e] = slope;
                const float u = GATE == kGateFirst ? x[c][e] * gate : x[c][e];
                us[c] = __builtin_fmaf(u, u, us[c]);
                if constexpr (PRE) {
                    hh = __builtin_fmaf(h[c][e], h[c][e], hh);
                    gh = __builtin_fmaf(dy[c][e] * w_pre[e], h[c][e], gh);
                }
            }
            uu += us[c];
        }
        if (PRE || whole) {
            constexpr int N = LANES < 64 ? LANES : 64;
            if (PRE) hh = sum_lanes(hh, N), gh = sum_lanes(gh, N);
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
        const float r2 = PRE ? rsqrt_fine(hh * inv_d + p.eps) : 1.0f;
        const float k2 = gh * inv_d * r2 * r2;
        // x becomes u, dy the gradient of u / rms(u) and, behind the second sums, of u
        float gu = 0.0f, r1[CH], part[CH];
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            r1[c] = !p.post ? 1.0f : rsqrt_fine((whole ? uu : sum_lanes(us[c], head_lanes)) * inv_n + p.eps);
            float dz[8], w_post[8], alpha[8], w_pre[8];
            weight(kPost, c, w_post);
            weight(kAlpha, c, alpha);
            if constexpr (PRE) weight(kPre, c, w_pre);
            part[c] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float t = up[c][e];
                if constexpr (PRE) {
                    t = __builtin_fmaf(r2, __builtin_fmaf(dy[c][e], w_pre[e], -h[c][e] * k2), t);
                    sum[2][c][e] = __builtin_fmaf(dy[c][e], h[c][e] * r2, sum[2][c][e]);
                } else {
                    t += dy[c][e];
                }
                up[c][e] = t;
                [[maybe_unused]] float gate, slope;
                if constexpr (GATE != kNoGate) gate_at(c, e, gate, slope);
                const float u = GATE == kGateFirst ? x[c][e] * gate : x[c][e];
                const float ur = u * r1[c], n = ur * w_post[e];
                sum[1][c][e] = __builtin_fmaf(t, GATE == kGateLast ? n * gate : n, sum[1][c][e]);
                float g = t * alpha[e];
                if constexpr (GATE == kGateLast) {
                    dz[e] = g * n * slope;
                    g *= gate;
                }
                sum[0][c][e] = __builtin_fmaf(g, ur, sum[0][c][e]);
                dy[c][e] = g * w_post[e];
                part[c] = __builtin_fmaf(dy[c][e], u, part[c]);
            }
            if (col < p.d) {
                if (p.dres) store8(static_cast<T*>(p.dres) + base + col, up[c]);
                if (GATE == kGateLast && p.dz) store8(static_cast<T*>(p.dz) + row * p.ld_z + col, dz);
            }
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
                [[maybe_unused]] float gate, slope;
                if constexpr (GATE == kGateFirst) gate_at(c, e, gate, slope);
                const float u = GATE == kGateFirst ? x[c][e] * gate : x[c][e];
                // (without the norm there is no u in it: an infinite one would leave NaN)
                float g = p.post ? r1[c] * __builtin_fmaf(-u, k1, dy[c][e]) : dy[c][e];
                if constexpr (GATE == kGateFirst) {
                    dz[e] = g * x[c][e] * slope;
                    g *= gate;
                }
                dy[c][e] = g;
            }
            if (GATE == kGateFirst && p.dz) store8(static_cast<T*>(p.dz) + row * p.ld_z + col, dz);
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
            if (sub == 0 && col < p.d && !(k == 0 && p.head)) store8(p.part[k] + static_cast<size_t>(blockIdx.x) * p.d + col, sum[k][c]);
        }
    }
    // a weight that the row's heads share: its sums over them here (joined with the workgroups' they took 22 us
    // for 16 heads of 128, 32768 rows, where the join takes 4)
    if (p.part[0] && p.head) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int col = (c * LANES + l) * kPiece;
            if (sub == 0 && col < p.d) {
#pragma unroll
                for (int e = 0; e < 8; e++) red[col + e] = sum[0][c][e];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.head; i += THREADS) {
            double s = 0.0;
            for (int at = i; at < p.d; at += p.head) s += red[at];
            p.part[0][static_cast<size_t>(blockIdx.x) * p.head + i] = static_cast<float>(s);
        }
    }
}

// The backward holds five rows: one piece a lane up to 4096 columns.
int bwd_lanes(int d) {
    const int pieces = d / kPiece;
    return pieces <= 256 ? gate_lanes(d) : pieces <= 384 ? 384 : pieces <= 1024 ? 512 : 1024;
}
template <class F>
hipError_t by_width_bwd(int d, F&& f) {
    using std::integral_constant;
    constexpr integral_constant<int, 1> one;
    constexpr integral_constant<int, 2> two;
    switch (bwd_lanes(d)) {
        case 8: return f(integral_constant<int, 8>{}, one);
        case 16: return f(integral_constant<int, 16>{}, one);
        case 32: return f(integral_constant<int, 32>{}, one);
        case 64: return f(integral_constant<int, 64>{}, one);
        case 128: return f(integral_constant<int, 128>{}, one);
        case 192: return f(integral_constant<int, 192>{}, one);
        case 256: return f(integral_constant<int, 256>{}, one);
        case 384: return f(integral_constant<int, 384>{}, one);
        case 1024: return f(integral_constant<int, 1024>{}, two);
    }
    return d / kPiece <= 512 ? f(integral_constant<int, 512>{}, one) : f(integral_constant<int, 512>{}, two);
}
template <class F>
hipError_t by_type(const la_gate_norm_config& c, F&& f) {
    return c.x_dtype == LA_BF16 ? f(uint16_t{}) : f(float{});
}
template <class F>
hipError_t by_mode(const la_gate_norm_config& c, F&& f) {
    using std::integral_constant;
    const GateAt at = c.gate == LA_GATE_NONE ? kNoGate : c.gate_first ? kGateFirst : kGateLast;
    auto gate = [&](auto g) { return c.pre ? f(g, std::true_type{}) : f(g, std::false_type{}); };
    if (at == kNoGate) return gate(integral_constant<GateAt, kNoGate>{});
    if (at == kGateLast) return gate(integral_constant<GateAt, kGateLast>{});
    return gate(integral_constant<GateAt, kGateFirst>{});
}

// A workgroup walks at most this many rows (each of its groups of lanes): what their FP32 sums may lose.
constexpr int kWalk = 128;

// Workgroups: all that are resident, or whole rounds of those where they would walk further.
int bwd_groups(const la_gate_norm_config& c) {
    const int lanes = bwd_lanes(c.d), rpw = lanes <= 64 ? 256 / lanes : 1;
    const int need = (c.rows + rpw - 1) / rpw, most = 256 * groups_for(lanes, c.gate != LA_GATE_NONE && c.pre);
    return need < most ? need : (need + most * kWalk - 1) / (most * kWalk) * most;
}

// The parameters' sums over the workgroups, in double and in a fixed order: 32 columns a workgroup, 32
// interleaved partial sums.
struct Joins {
    const float* part[3];
    float* out[3];
    int cols[3];
};
__global__ __launch_bounds__(1024) void join_kernel(Joins j, int parts) {
    __shared__ double red[32][33];
    const int k = blockIdx.y, l = threadIdx.x & 31, q = threadIdx.x >> 5, col = blockIdx.x * 32 + l;
    if (!j.out[k] || static_cast<int>(blockIdx.x) * 32 >= j.cols[k]) return;
    const bool in = col < j.cols[k];
    double s = 0.0;
    if (in) {
#pragma unroll 8
        for (int p = q; p < parts; p += 32) s += j.part[k][static_cast<size_t>(p) * j.cols[k] + col];
    }
    red[q][l] = s;
    __syncthreads();
    if (q == 0 && in) {
        s = 0.0;
#pragma unroll
        for (int i = 0; i < 32; i++) s += red[i][l];
        j.out[k][col] = static_cast<float>(s);
    }
}

}  // namespace

size_t gate_bwd_workspace(const la_gate_norm_config& c) {
    return static_cast<size_t>(bwd_groups(c)) * c.d * sizeof(float) * 3;
}

hipError_t launch_gate_bwd(const la_gate_norm_config& c, const GateArgs& a, hipStream_t s) {
    const int groups = bwd_groups(c);
    const size_t one = static_cast<size_t>(groups) * c.d;
    float* const part[3] = {a.dw_post ? a.part : nullptr, a.dalpha ? a.part + one : nullptr, a.dw_pre ? a.part + 2 * one : nullptr};
    if (groups > 0) {
        const GateBwd p{c.rows, c.d, c.head, c.gate, c.post, c.w_dtype, c.out_dtype, c.eps,
                        c.ld_x ? c.ld_x : c.d, c.ld_z ? c.ld_z : c.d, a.x, a.z, a.w_post, a.alpha, a.h, a.w_pre, a.dy, a.dh,
                        a.dx, a.dz, a.dres, {part[0], part[1], part[2]}};
        const hipError_t e = by_type(c, [&](auto t) {
            return by_mode(c, [&](auto gate, auto pre) {
                return by_width_bwd(c.d, [&](auto lanes, auto ch) {
                    constexpr int LANES = decltype(lanes)::value;
                    gate_bwd_kernel<decltype(t), LANES, decltype(ch)::value, decltype(gate)::value, decltype(pre)::value>
                        <<<groups, LANES <= 64 ? 256 : LANES, 0, s>>>(p);
                    return hipGetLastError();
                });
            });
        });
        if (e != hipSuccess) return e;
    }
    if (!a.dw_post && !a.dalpha && !a.dw_pre) return hipSuccess;
    const Joins j{{part[0], part[1], part[2]}, {a.dw_post, a.dalpha, a.dw_pre}, {c.head ? c.head : c.d, c.d, c.d}};
    join_kernel<<<dim3(static_cast<unsigned>((c.d + 31) / 32), 3), 1024, 0, s>>>(j, groups);
    return hipGetLastError();
}

}  // namespace la
