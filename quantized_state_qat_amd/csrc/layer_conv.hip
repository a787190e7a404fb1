// Depthwise causal convolution of width 2..4 with optional SiLU: forward, backward, one token.
//
// pre[t] = bias + sum_j w[j] z[t + j] over the rows z = state0 ++ x of a sequence.  A few
// multiplies and one exponential an element: memory bound.  A lane owns 16 bytes of channels
// (8 bf16, 4 fp32) and walks a few consecutive tokens with the window in registers, so each
// row is read once (plus W - 1 rows at the walk's start, which its neighbour has just read);
// the weights stay in registers.  A walk's first rows are fetched before anything else, ahead of
// the search for their sequence in a packing (98 -> 83 us) and of the window, in the backward
// always four tokens ahead (5% less).
//
// bf16, C = 2304, W = 4, SiLU: 8 sequences of 4096 tokens forward 61 us (5.4 TB/s), backward 107 us
// (4.8 TB/s, the vector units 67% busy) and 5 us for the parameters' sums; 40686 tokens in 64
// packed sequences 84 us (5.0 TB/s), their backward 162 us; one token of 256 sequences 5.6 us,
// launch and latencies.
#include "la_layer.hpp"

namespace la {
namespace {

// The channels' weights of one lane, widened.
template <int E, int W>
struct Taps {
    float w[W][E];
    float bias[E];
    // E W weights from c0 W on and E biases, in 16- or 8-byte pieces (c0 is a multiple of E).
    __device__ __forceinline__ void load(const void* wp, const void* bp, int dtype, int c0) {
        if (dtype == LA_BF16) load_as<uint16_t>(wp, bp, c0);
        else load_as<float>(wp, bp, c0);
    }
    template <class P>
    __device__ __forceinline__ void load_as(const void* wp, const void* bp, int c0) {
        constexpr int V = 8 / sizeof(P);  // elements of 8 bytes
        const uv2* w8 = reinterpret_cast<const uv2*>(static_cast<const P*>(wp) + static_cast<size_t>(c0) * W);
        uv2 raw[E * W / V], rb[E / V] = {};
#pragma unroll
        for (int i = 0; i < E * W / V; i++) raw[i] = w8[i];
        if (bp) {
#pragma unroll
            for (int i = 0; i < E / V; i++) rb[i] = reinterpret_cast<const uv2*>(static_cast<const P*>(bp) + c0)[i];
        }
        auto at = [](const uv2* r, int i) {
            if constexpr (sizeof(P) == 4) return __uint_as_float(r[i / 2][i % 2]);
            else return (i & 1) ? hi16(r[i / 4][i % 4 / 2]) : lo16(r[i / 4][i % 4 / 2]);
        };
#pragma unroll
        for (int e = 0; e < E; e++) {
#pragma unroll
            for (int j = 0; j < W; j++) w[j][e] = at(raw, e * W + j);
            bias[e] = at(rb, e);
        }
    }
};

template <class T>
struct ConvGeom {
    int B, T_, C, ldx, ldy, w_dtype, per, blocks;  // per: tokens a lane walks; blocks: token blocks per sequence
    const int32_t* cu;
};

// E elements of a row: 16 bytes, or 8 for four bf16.
template <class T, int E>
struct Piece {
    using Raw = std::conditional_t<sizeof(T) * E == 16, uv4, uv2>;
    static __device__ __forceinline__ Raw load(const T* p) { return *reinterpret_cast<const Raw*>(p); }
    static __device__ __forceinline__ void widen(Raw r, float (&v)[E]) {
        if constexpr (sizeof(T) * E == 16) {
            la::widen(r, v);
        } else {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                v[2 * i] = lo16(r[i]);
                v[2 * i + 1] = hi16(r[i]);
            }
        }
    }
    static __device__ __forceinline__ void store(T* p, const float (&v)[E]) {
        if constexpr (sizeof(T) * E == 16) store16(p, narrow(v));
        else *reinterpret_cast<uv2*>(p) = uv2{pack16(v[0], v[1]), pack16(v[2], v[3])};
    }
};

// Row `pos` (>= -(W-1)) of sequence b, from x or from the state before it.
template <class T, int W, int E>
__device__ __forceinline__ void conv_row_e(const T* x, const T* s0, int64_t begin, int pos, int b, int C, int ldx, int c0, float (&v)[E]) {
    if (pos >= 0) Piece<T, E>::widen(Piece<T, E>::load(x + (begin + pos) * ldx + c0), v);
    else if (s0) Piece<T, E>::widen(Piece<T, E>::load(s0 + (static_cast<int64_t>(b) * (W - 1) + (pos + W - 1)) * C + c0), v);
    else {
#pragma unroll
        for (int e = 0; e < E; e++) v[e] = 0.0f;
    }
}
template <class T, int W>
__device__ __forceinline__ uv4 conv_row(const T* x, const T* s0, int64_t begin, int pos, int b, int C, int ldx, int c0) {
    if (pos >= 0) return load16(x + (begin + pos) * ldx + c0);
    if (!s0) return uv4{0, 0, 0, 0};
    return load16(s0 + (static_cast<int64_t>(b) * (W - 1) + (pos + W - 1)) * C + c0);
}

template <class T, int W, int ACT>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvGeom<T> g, const T* __restrict__ x, const void* w,
                                                       const void* bias, const T* __restrict__ s0, T* __restrict__ y,
                                                       T* __restrict__ sT, int64_t items, int64_t main_blocks) {
    constexpr int E = Io<T>::kVec;
    const int nch = g.C / E;
    if (blockIdx.x >= main_blocks) {  // the last W - 1 rows of every sequence
        const int64_t i = (static_cast<int64_t>(blockIdx.x) - main_blocks) * 256 + threadIdx.x;
        if (i >= static_cast<int64_t>(g.B) * (W - 1) * nch) return;
        const int c0 = static_cast<int>(i % nch) * E;
        const int64_t r = i / nch;
        const int j = static_cast<int>(r % (W - 1)), b = static_cast<int>(r / (W - 1));
        Span sp{0, g.T_};
        if (g.cu) sp = packed_span(g.cu, b, g.T_);
        const int64_t begin = g.cu ? sp.begin : static_cast<int64_t>(b) * g.T_;
        const int len = sp.end - sp.begin;
        store16(sT + (static_cast<int64_t>(b) * (W - 1) + j) * g.C + c0,
                conv_row<T, W>(x, s0, begin, len + j - (W - 1), b, g.C, g.ldx, c0));
        return;
    }
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= items) return;
    const int c0 = static_cast<int>(i % nch) * E;
    const int64_t tb = i / nch;
    Taps<E, W> taps;
    taps.load(w, bias, g.w_dtype, c0);

    uv4 rows[8];
    auto fetch = [&](int64_t first, int n) {  // rows first .. first + n - 1 (up to eight)
#pragma unroll
        for (int k = 0; k < 8; k++) rows[k] = load16(x + (first + (k < n ? k : n - 1)) * g.ldx + c0);
    };
    // positions p0 .. p1 - 1 of sequence b, the first eight rows already fetched
    auto walk = [&](int64_t begin, int b, int p0, int p1) {
        float win[W][E];  // rows p - (W - 1) .. p
#pragma unroll
        for (int k = 0; k < W - 1; k++) widen(conv_row<T, W>(x, s0, begin, p0 - (W - 1) + k, b, g.C, g.ldx, c0), win[k + 1]);
        for (int p = p0; p < p1; p += 8) {
            if (p > p0) fetch(begin + p, p1 - p);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                if (p + k >= p1) break;
#pragma unroll
                for (int j = 0; j < W - 1; j++)
#pragma unroll
                    for (int e = 0; e < E; e++) win[j][e] = win[j + 1][e];
                widen(rows[k], win[W - 1]);
                float out[E];
#pragma unroll
                for (int e = 0; e < E; e++) {
                    float s = taps.bias[e];
#pragma unroll
                    for (int j = 0; j < W; j++) s = __builtin_fmaf(taps.w[j][e], win[j][e], s);
                    out[e] = ACT == LA_ACT_SILU ? s * sigmoid_for<T>(s) : s;
                }
                store16(y + (begin + p + k) * g.ldy + c0, narrow(out));
            }
        }
    };
    if (!g.cu) {
        const int b = static_cast<int>(tb / g.blocks);
        const int p0 = static_cast<int>(tb % g.blocks) * g.per;
        const int p1 = p0 + g.per < g.T_ ? p0 + g.per : g.T_;
        fetch(static_cast<int64_t>(b) * g.T_ + p0, p1 - p0);
        walk(static_cast<int64_t>(b) * g.T_, b, p0, p1);
        return;
    }
    int t = static_cast<int>(tb) * g.per;
    const int t1 = g.T_ - t < g.per ? g.T_ : t + g.per;
    fetch(t, t1 - t);  // in flight behind the search for their sequence
    for (const int t0 = t; t < t1;) {
        const int b = packed_find(g.cu, g.B, t);
        const Span sp = packed_span(g.cu, b, g.T_);
        if (t < sp.begin || t >= sp.end) {  // outside every sequence
            t++;
            continue;
        }
        const int stop = t1 < sp.end ? t1 : sp.end;
        if (t > t0) fetch(t, stop - t);
        walk(sp.begin, b, t - sp.begin, stop - sp.begin);
        t = stop;
    }
}

// dstate0: row j of z before x gets w[jj] dpre[j - jj] for jj <= j, and where the sequence is
// shorter than j the final state's own row passes through.
template <class T, int W, int ACT, int E>
__device__ __forceinline__ void conv_bwd_state(const ConvGeom<T>& g, const T* x, const void* w, const void* bias, const T* s0,
                                               const T* dy, const T* dsT, T* ds0, int b, int c0) {
    using Pc = Piece<T, E>;
    Span sp{0, g.T_};
    if (g.cu) sp = packed_span(g.cu, b, g.T_);
    const int64_t begin = g.cu ? sp.begin : static_cast<int64_t>(b) * g.T_;
    const int len = sp.end - sp.begin;
    Taps<E, W> taps;
    taps.load(w, bias, g.w_dtype, c0);
    float dp[W - 1][E];
#pragma unroll
    for (int p = 0; p < W - 1; p++) {
        float s[E], d[E] = {};
#pragma unroll
        for (int e = 0; e < E; e++) s[e] = taps.bias[e];
        if (p < len) {
#pragma unroll
            for (int j = 0; j < W; j++) {
                float r[E];
                conv_row_e<T, W>(x, s0, begin, p - (W - 1) + j, b, g.C, g.ldx, c0, r);
#pragma unroll
                for (int e = 0; e < E; e++) s[e] = __builtin_fmaf(taps.w[j][e], r[e], s[e]);
            }
            Pc::widen(Pc::load(dy + (begin + p) * g.ldy + c0), d);
        }
#pragma unroll
        for (int e = 0; e < E; e++) {
            if (ACT == LA_ACT_SILU) {
                const float sg = sigmoid_for<T>(s[e]);
                d[e] *= sg * __builtin_fmaf(s[e], 1.0f - sg, 1.0f);
            }
            dp[p][e] = p < len ? d[e] : 0.0f;
        }
    }
#pragma unroll
    for (int j = 0; j < W - 1; j++) {
        float out[E] = {};
        if (dsT && j >= len) Pc::widen(Pc::load(dsT + (static_cast<int64_t>(b) * (W - 1) + j - len) * g.C + c0), out);
#pragma unroll
        for (int jj = 0; jj <= j; jj++)
#pragma unroll
            for (int e = 0; e < E; e++) out[e] = __builtin_fmaf(taps.w[jj][e], dp[j - jj][e], out[e]);
        Pc::store(ds0 + (static_cast<int64_t>(b) * (W - 1) + j) * g.C + c0, out);
    }
}

// Backward.  dpre[t] = dy[t] act'(pre[t]); dz[u] = sum_j w[j] dpre[u - j] (+ dstate_T's row),
// dx the part of dz behind the state, dstate0 the part before; dw[j] = sum_t dpre[t] z[t + j].
// Work split as in the forward, 32 lanes of four channels by 8 token blocks a workgroup; each walk
// goes W - 1 tokens past its block for dpre there.  dw and dbias are summed over a lane's walks in
// registers in FP32, and in double over the workgroup in LDS and over workgroups (whose sums are
// FP32) by a second kernel: no atomics.
template <class T, int W, int ACT>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvGeom<T> g, const T* __restrict__ x, const void* w,
                                                       const void* bias, const T* __restrict__ s0,
                                                       const T* __restrict__ dy, const T* __restrict__ dsT,
                                                       T* __restrict__ dx, float* __restrict__ part, int64_t token_blocks,
                                                       T* ds0, int64_t main_blocks) {
    constexpr int E = 4;  // (with 8 bf16 a lane 232 registers left two waves a SIMD)
    using Pc = Piece<T, E>;
    const int nch = g.C / E;
    const int lane = threadIdx.x & 31, sub = threadIdx.x >> 5;
    const int ch = blockIdx.y * 32 + lane;
    const int c0 = ch * E;
    if (blockIdx.x >= main_blocks) {  // the initial states' gradients
        const int64_t b = (blockIdx.x - main_blocks) * 8 + sub;
        if (b < g.B && ch < nch) conv_bwd_state<T, W, ACT, E>(g, x, w, bias, s0, dy, dsT, ds0, static_cast<int>(b), c0);
        return;
    }
    float dw[W][E] = {}, db[E] = {};
    if (ch < nch) {
        Taps<E, W> taps;
        taps.load(w, bias, g.w_dtype, c0);
        auto walk = [&](int64_t begin, int len, int b, int p0, int p1) {
            typename Pc::Raw ax[4], ad[4];  // four tokens ahead
            auto fetch = [&](int p) {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int q = p + k < len ? p + k : len - 1;
                    ax[k] = Pc::load(x + (begin + q) * g.ldx + c0);
                    ad[k] = Pc::load(dy + (begin + q) * g.ldy + c0);
                }
            };
            fetch(p0);
            float win[W][E];
            float dp[W][E] = {};  // dpre of positions p - (W - 1) .. p
#pragma unroll
            for (int k = 0; k < W - 1; k++)
                conv_row_e<T, W>(x, s0, begin, p0 - (W - 1) + k, b, g.C, g.ldx, c0, win[k + 1]);
            const int pe = p1 + W - 1;
            // four tokens; EDGE: some of them behind the block or the sequence
            auto four = [&](int p, auto edge) {
                constexpr bool EDGE = decltype(edge)::value;
                typename Pc::Raw rx[4], rd[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    rx[k] = ax[k];
                    rd[k] = ad[k];
                }
                if (p + 4 < pe) fetch(p + 4);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int q = p + k;
                    if (EDGE && q >= pe) break;
#pragma unroll
                    for (int j = 0; j < W - 1; j++)
#pragma unroll
                        for (int e = 0; e < E; e++) {
                            win[j][e] = win[j + 1][e];
                            dp[j][e] = dp[j + 1][e];
                        }
                    float d[E];
                    Pc::widen(rx[k], win[W - 1]);
                    Pc::widen(rd[k], d);
                    const bool inside = !EDGE || q < len, mine = !EDGE || q < p1;
#pragma unroll
                    for (int e = 0; e < E; e++) {
                        float s = taps.bias[e];
#pragma unroll
                        for (int j = 0; j < W; j++) s = __builtin_fmaf(taps.w[j][e], win[j][e], s);
                        if (ACT == LA_ACT_SILU) {
                            const float sg = sigmoid_for<T>(s);
                            d[e] *= sg * __builtin_fmaf(s, 1.0f - sg, 1.0f);
                        }
                        dp[W - 1][e] = inside ? d[e] : 0.0f;
                        const float m = mine ? d[e] : 0.0f;
                        db[e] += m;
#pragma unroll
                        for (int j = 0; j < W; j++) dw[j][e] = __builtin_fmaf(m, mine ? win[j][e] : 0.0f, dw[j][e]);
                    }
                    const int u = q - (W - 1);  // its dx is now complete
                    if (u >= p0) {
                        float out[E] = {};
                        const int tail = u - len + W - 1;  // its row of the final state
                        if (EDGE && dsT && tail >= 0)
                            Pc::widen(Pc::load(dsT + (static_cast<int64_t>(b) * (W - 1) + tail) * g.C + c0), out);
#pragma unroll
                        for (int e = 0; e < E; e++)
#pragma unroll
                            for (int j = 0; j < W; j++)  // dz[u + W - 1 of z] = sum_j w[j] dpre[u + W - 1 - j]
                                out[e] = __builtin_fmaf(taps.w[j][e], dp[W - 1 - j][e], out[e]);
                        Pc::store(dx + (begin + u) * g.ldx + c0, out);
                    }
                }
            };
            int p = p0;
            for (; p + 4 <= p1 && p + 4 <= len; p += 4) four(p, std::false_type{});
            for (; p < pe; p += 4) four(p, std::true_type{});
        };
        for (int64_t tb = static_cast<int64_t>(blockIdx.x) * 8 + sub; tb < token_blocks; tb += main_blocks * 8) {
            if (!g.cu) {
                const int b = static_cast<int>(tb / g.blocks);
                const int p0 = static_cast<int>(tb % g.blocks) * g.per;
                const int p1 = g.T_ - p0 < g.per ? g.T_ : p0 + g.per;
                walk(static_cast<int64_t>(b) * g.T_, g.T_, b, p0, p1);
                continue;
            }
            int t = static_cast<int>(tb) * g.per;
            const int t1 = g.T_ - t < g.per ? g.T_ : t + g.per;
            while (t < t1) {
                const int b = packed_find(g.cu, g.B, t);
                const Span sp = packed_span(g.cu, b, g.T_);
                if (t < sp.begin || t >= sp.end) {  // outside every sequence: zero gradient
                    const float zero[E] = {};
                    Pc::store(dx + static_cast<int64_t>(t) * g.ldx + c0, zero);
                    t++;
                    continue;
                }
                const int stop = t1 < sp.end ? t1 : sp.end;
                walk(sp.begin, sp.end - sp.begin, b, t - sp.begin, stop - sp.begin);
                t = stop;
            }
        }
    }
    __shared__ float red[8][32][E + 1];
#pragma unroll
    for (int j = 0; j <= W; j++) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; e++) red[sub][lane][e] = j < W ? dw[j < W ? j : 0][e] : db[e];
        __syncthreads();
        const int tid = threadIdx.x;
        if (tid < 32 * E) {
            const int l = tid / E, e = tid % E, c = (blockIdx.y * 32 + l) * E + e;
            double s = 0.0;
#pragma unroll
            for (int k = 0; k < 8; k++) s += red[k][l][e];
            if (c < g.C) {
                const size_t at = static_cast<size_t>(blockIdx.x) * g.C * (W + 1) + (j < W ? static_cast<size_t>(c) * W + j
                                                                                          : static_cast<size_t>(g.C) * W + c);
                part[at] = static_cast<float>(s);
            }
        }
    }
}

template <class T, int W, int ACT>
__global__ __launch_bounds__(256) void conv_step_kernel(int B, int C, int ldx, int ldy, int w_dtype, const T* x, const void* w,
                                                        const void* bias, T* state, const int32_t* slots, int n_slots, T* y) {
    constexpr int E = Io<T>::kVec;
    const int nch = C / E;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<int64_t>(B) * nch) return;
    const int c0 = static_cast<int>(i % nch) * E, b = static_cast<int>(i / nch);
    const int slot = slots ? slots[b] : b;
    if (slots && (slot <= 0 || slot >= n_slots)) {  // padding
        store16(y + static_cast<int64_t>(b) * ldy + c0, uv4{0, 0, 0, 0});
        return;
    }
    T* st = state + static_cast<int64_t>(slot) * (W - 1) * C + c0;
    uv4 rows[W];
#pragma unroll
    for (int j = 0; j < W - 1; j++) rows[j] = load16(st + static_cast<int64_t>(j) * C);
    rows[W - 1] = load16(x + static_cast<int64_t>(b) * ldx + c0);
    Taps<E, W> taps;
    taps.load(w, bias, w_dtype, c0);
    float out[E];
#pragma unroll
    for (int e = 0; e < E; e++) out[e] = taps.bias[e];
#pragma unroll
    for (int j = 0; j < W; j++) {
        float r[E];
        widen(rows[j], r);
#pragma unroll
        for (int e = 0; e < E; e++) out[e] = __builtin_fmaf(taps.w[j][e], r[e], out[e]);
    }
    if (ACT == LA_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < E; e++) out[e] *= sigmoid_for<T>(out[e]);
    }
    store16(y + static_cast<int64_t>(b) * ldy + c0, narrow(out));
#pragma unroll
    for (int j = 0; j < W - 1; j++) store16(st + static_cast<int64_t>(j) * C, rows[j + 1]);
}

__global__ __launch_bounds__(1024) void reduce_parts_kernel(const float* __restrict__ part, int parts, int cols,
                                                            float* __restrict__ out, int split, float* __restrict__ out2) {
    __shared__ double red[32][33];
    const int l = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + l;
    double s = 0.0;
    if (col < cols) {
#pragma unroll 4
        for (int p = q; p < parts; p += 32) s += part[static_cast<size_t>(p) * cols + col];
    }
    red[q][l] = s;
    __syncthreads();
    if (q == 0 && col < cols) {
        s = 0.0;
#pragma unroll
        for (int k = 0; k < 32; k++) s += red[k][l];
        if (col < split) out[col] = static_cast<float>(s);
        else if (out2) out2[col - split] = static_cast<float>(s);
    }
}

template <class T>
__global__ __launch_bounds__(256) void zero_rows_kernel(T* out, int64_t n, int64_t width, int64_t ld) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
        out[i / width * ld + i % width] = T{};
}

// Tokens a lane walks in the backward: 32 where that still gives every CU several workgroups,
// fewer for short inputs.
int conv_bwd_per(const la_conv_config& c) {
    const int64_t tokens = static_cast<int64_t>(c.B) * c.T;  // an upper bound for a packing
    const int64_t lanes = (c.C / 4 + 31) / 32;
    int per = 32;
    while (per > 4 && lanes * (tokens / (8 * per)) < 512) per >>= 1;
    return per;
}

struct ConvBlocks {
    int64_t blocks;  // token blocks of the whole call
    int per_seq;     // token blocks a sequence (dense)
};
ConvBlocks conv_blocks(const la_conv_config& c, bool packed, int per) {
    const int n = (c.T + per - 1) / per;
    return {packed ? n : static_cast<int64_t>(n) * c.B, n};
}

template <class F>
hipError_t dispatch(const la_conv_config& c, F&& f) {
    auto act = [&](auto t, auto w) {
        if (c.act == LA_ACT_SILU) return f(t, w, std::integral_constant<int, LA_ACT_SILU>{});
        return f(t, w, std::integral_constant<int, LA_ACT_NONE>{});
    };
    auto width = [&](auto t) {
        switch (c.width) {
            case 2: return act(t, std::integral_constant<int, 2>{});
            case 3: return act(t, std::integral_constant<int, 3>{});
            default: return act(t, std::integral_constant<int, 4>{});
        }
    };
    if (c.x_dtype == LA_BF16) return width(uint16_t{});
    return width(float{});
}

template <class T>
ConvGeom<T> geom(const la_conv_config& c, const int32_t* cu, int per, int blocks) {
    return {c.B, c.T, c.C, c.ld_x ? c.ld_x : c.C, c.ld_y ? c.ld_y : c.C, c.w_dtype, per, blocks, cu};
}

}  // namespace

hipError_t launch_conv_fwd(const la_conv_config& c, const ConvArgs& a, hipStream_t s) {
    return dispatch(c, [&](auto t, auto w, auto act) {
        using T = decltype(t);
        constexpr int W = decltype(w)::value, ACT = decltype(act)::value;
        const int nch = c.C / Io<T>::kVec;
        int per = 16;
        while (per > 1 && (static_cast<int64_t>(a.cu ? 1 : c.B) * c.T / per) * nch < 65536) per >>= 1;
        const ConvBlocks nb = conv_blocks(c, a.cu != nullptr, per);
        const int64_t items = nb.blocks * nch, main_blocks = (items + 255) / 256;
        const int64_t extra = a.sT ? (static_cast<int64_t>(c.B) * (W - 1) * nch + 255) / 256 : 0;
        if (main_blocks + extra == 0) return hipSuccess;
        conv_fwd_kernel<T, W, ACT><<<dim3(static_cast<unsigned>(main_blocks + extra)), 256, 0, s>>>(
            geom<T>(c, a.cu, per, nb.per_seq), static_cast<const T*>(a.x), a.w, a.bias, static_cast<const T*>(a.s0),
            static_cast<T*>(a.y), static_cast<T*>(a.sT), items, main_blocks);
        return hipGetLastError();
    });
}

// Workgroups along the tokens, each with its partial sums: one for eight token blocks, and no more
// than 8192 over all channels (32 a CU), beyond which each takes several.
int64_t conv_bwd_parts(const la_conv_config& c, int64_t blocks) {
    const int64_t lanes = (c.C / 4 + 31) / 32, cap = 8192 / lanes > 1 ? 8192 / lanes : 1;
    return (blocks + 7) / 8 < cap ? (blocks + 7) / 8 : cap;
}

size_t conv_bwd_workspace(const la_conv_config& c) {  // (a packing has fewer blocks)
    const int64_t parts = conv_bwd_parts(c, conv_blocks(c, false, conv_bwd_per(c)).blocks);
    return static_cast<size_t>(parts) * c.C * (c.width + 1) * sizeof(float);
}

hipError_t launch_conv_bwd(const la_conv_config& c, const ConvArgs& a, hipStream_t s) {
    return dispatch(c, [&](auto t, auto w, auto act) {
        using T = decltype(t);
        constexpr int W = decltype(w)::value, ACT = decltype(act)::value;
        const int per = conv_bwd_per(c);
        const ConvBlocks nb = conv_blocks(c, a.cu != nullptr, per);
        const ConvGeom<T> g = geom<T>(c, a.cu, per, nb.per_seq);
        // (no sequences, or no tokens: no parts, and the sums below are zero)
        const int64_t gy = c.B > 0 ? conv_bwd_parts(c, nb.blocks) : 0, extra = a.ds0 ? (c.B + 7) / 8 : 0;
        if (gy + extra > 0)
            conv_bwd_kernel<T, W, ACT><<<dim3(static_cast<unsigned>(gy + extra), (c.C / 4 + 31) / 32), 256, 0, s>>>(
                g, static_cast<const T*>(a.x), a.w, a.bias, static_cast<const T*>(a.s0), static_cast<const T*>(a.dy),
                static_cast<const T*>(a.dsT), static_cast<T*>(a.dx), a.part, nb.blocks, static_cast<T*>(a.ds0), gy);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess && c.B == 0 && a.cu)  // every token is outside every sequence
            e = launch_zero_rows(a.dx, c.x_dtype, c.T, c.C, g.ldx, s);
        if (e != hipSuccess) return e;
        return launch_reduce_parts(a.part, static_cast<int>(gy), c.C * (W + 1), a.dw, c.C * W, a.dbias, s);
    });
}

hipError_t launch_conv_step(const la_conv_config& c, const ConvArgs& a, hipStream_t s) {
    return dispatch(c, [&](auto t, auto w, auto act) {
        using T = decltype(t);
        constexpr int W = decltype(w)::value, ACT = decltype(act)::value;
        const int64_t items = static_cast<int64_t>(c.B) * (c.C / Io<T>::kVec);
        conv_step_kernel<T, W, ACT><<<dim3(static_cast<unsigned>((items + 255) / 256)), 256, 0, s>>>(
            c.B, c.C, c.ld_x ? c.ld_x : c.C, c.ld_y ? c.ld_y : c.C, c.w_dtype, static_cast<const T*>(a.x), a.w, a.bias,
            static_cast<T*>(a.state), a.slots, a.n_slots, static_cast<T*>(a.y));
        return hipGetLastError();
    });
}

hipError_t launch_reduce_parts(const float* part, int parts, int cols, float* out, int split, float* out2,
                               hipStream_t s) {
    if (cols == 0) return hipSuccess;
    reduce_parts_kernel<<<dim3((cols + 31) / 32), 1024, 0, s>>>(part, parts, cols, out, split, out2);
    return hipGetLastError();
}

hipError_t launch_zero_rows(void* out, int dtype, int64_t rows, int64_t width, int64_t ld, hipStream_t s) {
    const int64_t n = rows * width;
    if (!out || n == 0) return hipSuccess;
    const unsigned grid = static_cast<unsigned>(n < 65536 * 256 ? (n + 255) / 256 : 65536);
    if (dtype == LA_BF16) zero_rows_kernel<<<grid, 256, 0, s>>>(static_cast<uint16_t*>(out), n, width, ld);
    else zero_rows_kernel<<<grid, 256, 0, s>>>(static_cast<float*>(out), n, width, ld);
    return hipGetLastError();
}

}  // namespace la
