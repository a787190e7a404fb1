// The selective scan in chunks of 64 tokens: shared pieces of its forward and backward.
//
// With cum_t the chunk's cumulative log decay (its own token included), Delta_s the step,
//     G = C B^T,  L_ts = exp(cum_t - cum_s) for s <= t (else 0),  M_ts = G_ts L_ts Delta_s
//     Y = M X + diag(exp cum) (C S)            S: the state entering the chunk
//     S_end = exp(cum_end) S + (W B)^T X       W_s = exp(cum_end - cum_s) Delta_s
// Every product runs on the matrix cores as 16 x 16 tiles with 32 values of the contraction at
// a time.  bf16 inputs enter them as they are; an operand formed in FP32 (M, the state, W X) is
// written as a sum of bf16 parts, so that products keep FP32's precision (three parts: 24 bits)
// or 16 bits (two parts) where a bf16 result takes the sum.  FP32 inputs run on the FP32 matrix
// instruction, eight contraction steps of four values, in the same lane layout.
#pragma once

#include "la_layer.hpp"
#include "la_mfma.hpp"

namespace la {

constexpr int kQ = 64;   // tokens a chunk
constexpr int kPT = 64;  // value columns a workgroup

// LDS row of n elements.  bf16: 32 bytes over a multiple of 256 or 64 (288, 160, 96) for rows that
// are read in 16-byte pieces (8.3 cycles a kilobyte against 9.5 at 16 bytes over), 144 bytes for
// the 64-wide rows that are also written in 8-byte pieces (10 cycles against 17).  Two 8-byte reads
// or transposed reads take 17 cycles a kilobyte at any of these, so a row operand is always one
// 16-byte piece a lane.
template <class T>
constexpr int lds_row(int n) {
    return sizeof(T) == 2 ? (n == 128 ? 144 : n == 64 ? 80 : 48) : n + 4;
}
template <class T>
constexpr int lds_row64() {
    return sizeof(T) == 2 ? 72 : 68;
}

// State rows in the accumulators: register r of tile i in lane group g is row state_n(i, 4 g + r),
// so that two tiles hold the eight consecutive rows of a lane's operand piece.
__device__ __forceinline__ int state_n(int i, int m) { return 32 * (i >> 1) + 8 * (m >> 2) + 4 * (i & 1) + (m & 3); }

template <class T>
struct Mat;

template <>
struct Mat<uint16_t> {
    typedef bf8 Frag;
    template <int P>
    static constexpr int parts = P;
    static __device__ __forceinline__ f4 mma(Frag a, Frag b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // Row operand: 8 consecutive elements from k (lane group g: k = 32 i + 8 g).
    static __device__ __forceinline__ Frag row8(const uint16_t* p) { return *reinterpret_cast<const bf8*>(p); }
    // Column operand: rows r0 + 8 g .. + 7 of column c0 + lane % 16, by two transposed reads (in
    // each 16 lanes, lane 4 j + q addresses row j's 8 bytes q and lane i receives column i).
    static __device__ __forceinline__ Frag tr8(const uint16_t* p, int stride) {
        const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p));
        const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 4 * stride));
        return __builtin_bit_cast(Frag, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ Frag col8(const uint16_t* base, int stride, int r0, int c0, int lane) {
        const int i = lane & 15, g = lane >> 4;
        return tr8(base + (r0 + 8 * g + (i >> 2)) * stride + c0 + 4 * (i & 3), stride);
    }
    // The same of column state_n(tile, lane % 16).
    static __device__ __forceinline__ Frag col8_state(const uint16_t* base, int stride, int r0, int tile, int lane) {
        const int i = lane & 15, g = lane >> 4;
        return tr8(base + (r0 + 8 * g + (i >> 2)) * stride + state_n(tile, 4 * (i & 3)), stride);
    }
    static __device__ __forceinline__ void widen8(Frag f, float (&v)[8]) { widen(__builtin_bit_cast(uv4, f), v); }
    // x = sum of the P parts (P = 2: to 2^-17 of x; P = 3: exactly).
    template <int P>
    static __device__ __forceinline__ void split(const float (&x)[8], Frag (&out)[P]) {
        uv4 w[P];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
            for (int k = 0; k < P; k++) {
                w[k][i] = pack16(a, b);
                if (k + 1 < P) {
                    a -= lo16(w[k][i]);
                    b -= hi16(w[k][i]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < P; k++) out[k] = __builtin_bit_cast(Frag, w[k]);
    }
    // Four values as P planes of 8 bytes.
    template <int P>
    static __device__ __forceinline__ void put4(uint16_t* p, int plane, const float (&x)[4]) {
        float v[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 0; k < P; k++) {
            const uint32_t a = pack16(v[0], v[1]), b = pack16(v[2], v[3]);
            *reinterpret_cast<uv2*>(p + k * plane) = uv2{a, b};
            if (k + 1 < P) {
                v[0] -= lo16(a);
                v[1] -= hi16(a);
                v[2] -= lo16(b);
                v[3] -= hi16(b);
            }
        }
    }
    static __device__ __forceinline__ void get4(const uint16_t* p, float (&v)[4]) {
        const uv2 a = *reinterpret_cast<const uv2*>(p);
        v[0] = lo16(a[0]);
        v[1] = hi16(a[0]);
        v[2] = lo16(a[1]);
        v[3] = hi16(a[1]);
    }
};

template <>
struct Mat<float> {
    typedef f8 Frag;
    template <int P>
    static constexpr int parts = 1;
    static __device__ __forceinline__ f4 mma(Frag a, Frag b, f4 c) {
#pragma unroll
        for (int j = 0; j < 8; j++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Frag two(const float* p, const float* q) {
        const f4 a = *reinterpret_cast<const f4*>(p), b = *reinterpret_cast<const f4*>(q);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    static __device__ __forceinline__ Frag row8(const float* p) { return two(p, p + 4); }
    static __device__ __forceinline__ Frag col8(const float* base, int stride, int r0, int c0, int lane) {
        const float* p = base + (r0 + 8 * (lane >> 4)) * stride + c0 + (lane & 15);
        Frag f;
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = p[j * stride];
        return f;
    }
    static __device__ __forceinline__ Frag col8_state(const float* base, int stride, int r0, int tile, int lane) {
        return col8(base, stride, r0, state_n(tile, lane & 15) - (lane & 15), lane);
    }
    static __device__ __forceinline__ void widen8(Frag f, float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = f[j];
    }
    template <int P>
    static __device__ __forceinline__ void split(const float (&x)[8], Frag (&out)[P]) {
        static_assert(P == 1, "FP32 operands have one part");
#pragma unroll
        for (int j = 0; j < 8; j++) out[0][j] = x[j];
    }
    template <int P>
    static __device__ __forceinline__ void put4(float* p, int, const float (&x)[4]) {
        *reinterpret_cast<f4*>(p) = f4{x[0], x[1], x[2], x[3]};
    }
    static __device__ __forceinline__ void get4(const float* p, float (&v)[4]) {
        const f4 a = *reinterpret_cast<const f4*>(p);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = a[i];
    }
};

// x, as a value that the compiler knows nothing about.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Four values summed over the four rows of 16 lanes, lane row g left with value g's sum: three
// exchanges for what four whole sums take eight for.
__device__ __forceinline__ float rows_scatter4(const float (&v)[4]) {
    auto half = [](float a, float b) {  // lanes 0..31: a's sum over lane and lane + 32, lanes 32..63: b's
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    };
    const float x = half(v[0], v[2]), y = half(v[1], v[3]);
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 2^(hi + lo) for |lo| far below an ulp of hi.
__device__ __forceinline__ float exp2_two(float hi, float lo) {
    const float r = __builtin_amdgcn_exp2f(hi);
    return __builtin_fmaf(r, lo * 0.693147180559945309f, r);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t a = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xF, true);
    const uint32_t b = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xF, true);
    return __builtin_bit_cast(double, static_cast<uint64_t>(a) | (static_cast<uint64_t>(b) << 32));
}
// Inclusive prefix sum over the wave's 64 lanes: shifts within rows of 16, then the rows' totals.
__device__ __forceinline__ double wave_prefix(double x) {
    x += dpp_f64<0x111, 0xF>(x);
    x += dpp_f64<0x112, 0xF>(x);
    x += dpp_f64<0x114, 0xF>(x);
    x += dpp_f64<0x118, 0xF>(x);
    x += dpp_f64<0x142, 0xA>(x);  // lane 15 of each even row to the row after it
    x += dpp_f64<0x143, 0xC>(x);  // lane 31 to rows 2 and 3
    return x;
}
__device__ __forceinline__ double wave_last(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t a = __builtin_amdgcn_readlane(static_cast<int>(u), 63);
    const uint32_t b = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), 63);
    return __builtin_bit_cast(double, static_cast<uint64_t>(a) | (static_cast<uint64_t>(b) << 32));
}

// log(1 + exp(z)) = max(z, 0) + log1p(e), e = exp(-|z|) in (0, 1]; log1p(e) = 2 artanh(e / (2 + e)),
// the argument at most 1/3: its series to the 15th power is within 2^-26 of the sum.  A third of
// the library functions' instructions; one wave forms it while others wait.
__device__ __forceinline__ float softplus_fine(float z) {
    const float e = exp_fine(fmaxf(-fabsf(z), -87.0f));
    const float d = 2.0f + e, r = __builtin_amdgcn_rcpf(d);
    const float q = e * r;
    const float s = __builtin_fmaf(__builtin_fmaf(-d, q, e), r, q);
    const float x = s * s;
    float p = 1.0f / 15.0f;
    p = __builtin_fmaf(p, x, 1.0f / 13.0f);
    p = __builtin_fmaf(p, x, 1.0f / 11.0f);
    p = __builtin_fmaf(p, x, 1.0f / 9.0f);
    p = __builtin_fmaf(p, x, 1.0f / 7.0f);
    p = __builtin_fmaf(p, x, 1.0f / 5.0f);
    p = __builtin_fmaf(p, x, 1.0f / 3.0f);
    const float two_s = s + s;
    return (z < 0.0f ? 0.0f : z) + __builtin_fmaf(two_s * x, p, two_s);  // (NaN stays NaN)
}

// One chunk's decays for a head.  Exponents are in units of log2; the cumulative sums are formed
// in double and kept as hi + lo floats, so that the difference of two far into a long decay
// keeps FP32's relative precision.
struct Decay {
    float hi[kQ], lo[kQ];  // cum
    float delta[kQ];       // 0 behind the sequence
    float head[kQ];        // exp(cum_t)
    float tail[kQ];        // exp(cum_end - cum_t)
    float w[kQ];           // tail Delta
    float z[kQ];           // dt + dt_bias
    float total[kQ];       // [0]: exp(cum_end)
};
// By one whole wave, lane = token, from z (0 steps from token `live` on).  Returns cum_end (log2).
__device__ __forceinline__ double make_decay(Decay& d, float z, int softplus, int live, float A) {
    const int t = threadIdx.x & 63;
    const float delta = t < live ? (softplus ? softplus_fine(z) : z) : 0.0f;
    const double cum = wave_prefix(static_cast<double>(delta) * (static_cast<double>(A) * 1.4426950408889634));
    const double end = wave_last(cum);
    const float hi = static_cast<float>(cum), lo = static_cast<float>(cum - hi);
    const double rest = end - cum;
    const float rh = static_cast<float>(rest), rl = static_cast<float>(rest - rh);
    d.hi[t] = hi;
    d.lo[t] = lo;
    d.delta[t] = delta;
    d.head[t] = exp2_two(hi, lo);
    const float tail = exp2_two(rh, rl);
    d.tail[t] = tail;
    d.w[t] = tail * delta;
    d.z[t] = z;
    if (t == 63) d.total[0] = exp2_two(hi, lo);
    return end;
}
// A Decay on its way from memory to LDS, a few words a thread.
template <int THREADS>
struct DecayAhead {
    static constexpr int W = static_cast<int>(sizeof(Decay) / 4) / THREADS;
    uint32_t r[W];
    __device__ __forceinline__ void load(const Decay* from) {
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(from, sizeof(Decay));
#pragma unroll
        for (int i = 0; i < W; i++) r[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, static_cast<int>(threadIdx.x) * 4, i * THREADS * 4, 0);
    }
    __device__ __forceinline__ void store(Decay& to) const {
#pragma unroll
        for (int i = 0; i < W; i++) reinterpret_cast<uint32_t*>(&to)[threadIdx.x + i * THREADS] = r[i];
    }
};
// Eight consecutive values of one of the arrays (16-byte aligned).
__device__ __forceinline__ void get8(const float* a, float (&v)[8]) {
    const f4 x = *reinterpret_cast<const f4*>(a), y = *reinterpret_cast<const f4*>(a + 4);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[i] = x[i];
        v[4 + i] = y[i];
    }
}
// exp(cum_t - cum_s)
__device__ __forceinline__ float pair_decay(float thi, float tlo, float shi, float slo) {
    return __builtin_amdgcn_exp2f((thi - shi) + (tlo - slo));
}

// Launch parameters of the chunk kernels.
struct ScanP {
    int B, T, H, G, dk, dv, softplus, dt_dtype, out_dtype;
    int64_t ld_x, ld_b, ld_c, ld_dt;
    const int32_t* cu;
    const void* x;
    const void* dt;
    const float* A;
    const void* b;
    const void* c;
    const float* D;
    const float* bias;
};
inline ScanP scan_params(const la_scan_config& c, const ScanArgs& a) {
    return {c.B, c.T, c.H, c.G, c.d_k, c.d_v, c.softplus, c.dt_dtype, c.out_dtype,
            c.ld_x ? c.ld_x : static_cast<int64_t>(c.H) * c.d_v, c.ld_b ? c.ld_b : static_cast<int64_t>(c.G) * c.d_k,
            c.ld_c ? c.ld_c : static_cast<int64_t>(c.G) * c.d_k, c.ld_dt ? c.ld_dt : static_cast<int64_t>(c.H),
            a.cu, a.x, a.dt, a.A, a.b, a.c, a.D, a.bias};
}

// Token range of sequence b: rows begin .. begin + len - 1 of the tensors.
struct SeqRange {
    int64_t begin;
    int len;
};
__device__ __forceinline__ SeqRange seq_range(const ScanP& p, int b) {
    if (!p.cu) return {static_cast<int64_t>(b) * p.T, p.T};
    const Span s = packed_span(p.cu, b, p.T);
    return {s.begin, s.end - s.begin};
}

// dt of a chunk's tokens, lane = token: the word that holds it on its way (no branch around the
// load and nothing that would wait for it), and the value once it is needed.
struct DtAhead {
    uint32_t word = 0, half = 0;
    __device__ __forceinline__ void fetch(const ScanP& p, int64_t row0, int h, int lane, int live) {
        const int es = p.dt_dtype == LA_BF16 ? 2 : 4;
        const int64_t byte = (row0 * p.ld_dt + h) * es;
        const __amdgpu_buffer_rsrc_t r =
            make_rsrc(static_cast<const char*>(p.dt) + (byte & ~int64_t{3}), static_cast<size_t>(kQ) * p.ld_dt * es + 4);
        const uint32_t off = static_cast<uint32_t>((byte & 3) + lane * p.ld_dt * es);
        half = off & 2;
        word = __builtin_amdgcn_raw_buffer_load_b32(r, lane < live ? static_cast<int>(off & ~3u) : -4, 0, 0);
    }
    __device__ __forceinline__ float value(const ScanP& p) const {
        return p.dt_dtype == LA_F32 ? __uint_as_float(word) : half ? hi16(word) : lo16(word);
    }
};
// A [64][COLS] tile of rows `row0 ..` in registers and on its way to LDS: 16-byte pieces, the
// pieces of a row on neighbouring threads; rows from `live` on and columns from `cols` on are
// zero.  The buffer's bounds give the zeros: no branch around a load, so that the loads stay in
// flight behind the products of the chunk before.
template <class T, int COLS, int THREADS>
struct Tile {
    static constexpr int E = Io<T>::kVec;
    static constexpr int PPR = COLS / E;
    static constexpr int K = kQ * PPR / THREADS > 0 ? kQ * PPR / THREADS : 1;
    uv4 r[K];
    __device__ __forceinline__ void load(const T* base, int64_t ld, int live, int cols) {
        // (the offset of a row from `live` on is at least the buffer's size)
        const uint32_t bytes = static_cast<uint32_t>((live < kQ ? live : kQ) * ld * static_cast<int>(sizeof(T)));
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(base, bytes);
#pragma unroll
        for (int k = 0; k < K; k++) {
            const int i = threadIdx.x + THREADS * k;
            const int row = i / PPR, col = (i % PPR) * E;
            int off = (row * static_cast<int>(ld) + col) * static_cast<int>(sizeof(T));
            if (COLS == 32 && col >= cols) off = -16;  // d_k = 16 in a tile of 32
            if (kQ * PPR < THREADS && row >= kQ) off = -16;
            r[k] = __builtin_bit_cast(uv4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
        }
    }
    __device__ __forceinline__ void store(T* lds, int stride) const {
#pragma unroll
        for (int k = 0; k < K; k++) {
            const int i = threadIdx.x + THREADS * k;
            if (kQ * PPR < THREADS && i >= kQ * PPR) continue;
            store16(lds + (i / PPR) * stride + (i % PPR) * E, r[k]);
        }
    }
};

// Workgroups go round the eight dies in launch order: unit u of consecutive ones on one die,
// so that the heads that read the same b and c share its L2.
__device__ __forceinline__ uint32_t die_unit(uint32_t block, uint32_t blocks) {
    const uint32_t q = blocks / 8, r = blocks % 8, d = block % 8;
    return d * q + (d < r ? d : r) + block / 8;
}
// u modulo n, u divided by n: the result in scalar registers (the same in every lane).
__device__ __forceinline__ int take(uint32_t& u, int n) {
    const uint32_t q = u / static_cast<uint32_t>(n);
    const int r = __builtin_amdgcn_readfirstlane(static_cast<int>(u - q * n));
    u = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(q)));
    return r;
}

}  // namespace la
