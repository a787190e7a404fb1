// Straight-through gradients of the product of 8-bit codes: dx = (dy s_w) c_w, dweight = (dy s_x)^T c_x.
//
// Both are products on the FP16 matrix cores: FP16 holds every code exactly, and dy times the scale,
// brought to [2^14, 2^15) by a power of two for each row of the operand (scale_up), is off by at most
// 2^-22 of itself in two parts.  (One part, off by 2^-11, halves the product's work, but a bf16 result
// of terms that cancel shows it: such a gradient then differs from the formula's by more than its own rounding.)
// The products sum over an index that is not contiguous in what the caller holds (channels of dx,
// tokens of dweight), so a pass over dy and one over each matrix of codes lay the operands out first,
// 128 bytes of the summed index at a time: they move 2 to 8 bytes an element once where the product
// itself reads an operand many times over.  32768 x 2048 x 2048 from bf16 dy to bf16 dx and FP32 dweight 1145 to
// 1160 us: 41 + 41 + 112 laying out (3.5 to 6.0 TB/s: memory bound), 500 to 530 and 470 to 510 the products (1040 to
// 1170 TFLOP/s by the clock that a card's power leaves), 15 joining dweight's four parts.
#include "linear_gemm.hpp"

namespace la {
namespace {

__device__ __forceinline__ uint32_t finite_abs(float v) {
    const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
    return u < 0x7F800000u ? u : 0;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// 8 elements of a row from column n on, zeros from N on.  FULL: all are there, 16-byte aligned.
template <bool FULL, class T>
__device__ __forceinline__ void load_part(const T* row, int n, int N, float (&v)[8]) {
    if constexpr (FULL) {
        if constexpr (sizeof(T) == 2) widen(load16(row + n), v);
        else load_eight(row + n, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = n + e < N ? load_elem(row, n + e, sizeof(T) == 2 ? LA_BF16 : LA_F32) : 0.0f;
    }
}

struct DyArgs {
    const void* dy;
    const float* xs;
    const float* ws;
    int M, N, wide;
    int64_t ld;
    uint32_t* rowmax;  // [M] of |dy s_w|, or null
    uint32_t* colmax;  // [N] of |dy s_x|, or null
    float* part;       // [ceil(M / 64)][N], or null
    float* dbias;      // [N], or null
    char* qx;          // M rows of N in chunks of 64, or null
    char* qw;          // N rows of M, or null
};

// Largest magnitudes of rows and columns (integer maxima: their order does not matter) and the sums
// of 64 rows: a workgroup has 64 rows of 256 columns, eight of each a lane, all loaded together.  Floating maxima
// pass over NaN by themselves; where an infinity came up, the finite values' are taken in another pass.
// 32768 x 2048 bf16 40 us (3.3 TB/s; 39 without the columns' atomics, 43 with every value looked at for
// infinities).
template <bool FULL, class T>
__device__ __forceinline__ void stats_rows(const DyArgs& a, int m0, int n, int ty, float (&cs)[8], uint32_t (&cm)[8],
                                           uint32_t (&rows)[64]) {
    float ws[8] = {}, xs[8] = {}, v[8][8];
    if (a.rowmax) load_part<FULL>(a.ws, n, a.N, ws);
#pragma unroll
    for (int k = 0; k < 8; k++) {
        const int m = m0 + ty + 8 * k;
        if (FULL || m < a.M) {
            load_part<FULL>(static_cast<const T*>(a.dy) + m * a.ld, n, a.N, v[k]);
            if (a.colmax) xs[k] = a.xs[m];
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) v[k][e] = 0.0f;
        }
    }
    float rm[8] = {}, cf[8] = {}, top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            rm[k] = fmaxf(rm[k], fabsf(v[k][e] * ws[e]));
            cf[e] = fmaxf(cf[e], fabsf(v[k][e] * xs[k]));
            cs[e] += v[k][e];
        }
        top = fmaxf(top, rm[k]);
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
        cm[e] = __float_as_uint(cf[e]);
        top = fmaxf(top, cf[e]);
    }
#pragma unroll
    for (int k = 0; k < 8; k++) {
        const uint32_t r = __float_as_uint(group_max_abs<32>(rm[k]));
        if ((threadIdx.x & 31) == 0) rows[ty + 8 * k] = r;
    }
    if (!__any(top == __builtin_inff())) return;
#pragma unroll
    for (int e = 0; e < 8; e++) cm[e] = 0;
#pragma unroll 1
    for (int k = ty; k < 64 && m0 + k < a.M; k += 8) {
        load_part<FULL>(static_cast<const T*>(a.dy) + (m0 + k) * a.ld, n, a.N, v[0]);
        const float x = a.colmax ? a.xs[m0 + k] : 0.0f;
        uint32_t r = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            r = umax(r, finite_abs(v[0][e] * ws[e]));
            cm[e] = umax(cm[e], finite_abs(v[0][e] * x));
        }
        r = __float_as_uint(group_max_abs<32>(__uint_as_float(r)));
        if ((threadIdx.x & 31) == 0) rows[k] = r;
    }
}
template <class T>
__global__ __launch_bounds__(256) void stats_kernel(DyArgs a) {
    __shared__ float sum[8][256];
    __shared__ uint32_t top[8][256], rows[64];
    const int across = (a.N + 255) / 256;
    const int n0 = (blockIdx.x % across) * 256, m0 = (blockIdx.x / across) * 64;
    const int c = (threadIdx.x & 31) * 8, ty = threadIdx.x >> 5;
    float cs[8] = {};
    uint32_t cm[8] = {};
    if (a.wide && m0 + 64 <= a.M && n0 + 256 <= a.N) stats_rows<true, T>(a, m0, n0 + c, ty, cs, cm, rows);
    else stats_rows<false, T>(a, m0, n0 + c, ty, cs, cm, rows);
#pragma unroll
    for (int e = 0; e < 8; e++) {
        sum[ty][c + e] = cs[e];
        top[ty][c + e] = cm[e];
    }
    __syncthreads();
    if (a.rowmax && threadIdx.x < 64 && rows[threadIdx.x]) atomicMax(a.rowmax + m0 + threadIdx.x, rows[threadIdx.x]);
    const int col = n0 + threadIdx.x;
    if (col >= a.N) return;
    float s = 0.0f;
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; k++) {
        s += sum[k][threadIdx.x];
        m = umax(m, top[k][threadIdx.x]);
    }
    if (a.part) a.part[static_cast<int64_t>(blockIdx.x / across) * a.N + col] = s;
    if (a.colmax && m) atomicMax(a.colmax + col, m);
}

// A part is 64 elements = 128 bytes of the summed index; a row holds chunk c's parts beside each other.
constexpr int kParts = 1 << kShift;  // of dy times the scale
__device__ __forceinline__ int64_t part_at(int chunk, int part, int parts) { return (static_cast<int64_t>(chunk) * parts + part) * 128; }

// Eight scaled values as FP16 in two parts.  The second is what the first leaves, which an infinity
// leaves infinite: it meets the same codes.
__device__ __forceinline__ void store_parts(char* o, const float (&v)[8]) {
    hv8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        hi[e] = static_cast<_Float16>(v[e]);
        lo[e] = static_cast<_Float16>(v[e] - __builtin_amdgcn_fmed3f(static_cast<float>(hi[e]), -65504.0f, 65504.0f));
    }
    *reinterpret_cast<hv8*>(o) = hi;
    *reinterpret_cast<hv8*>(o + 128) = lo;
}

// 64 x 64 of dy into both operands: along the rows from registers, along the columns through LDS (110 us for
// 32768 x 2048 bf16, 678 MB, 6.0 TB/s).
template <bool FULL, class T>
__device__ __forceinline__ void lay_dy(const DyArgs& a, int cm, int cn, T (&tile)[64][66]) {
    const int n0 = cn * 64, m0 = cm * 64;
    const int64_t rowx = part_at((a.N + 63) / 64, 0, kParts), roww = part_at((a.M + 63) / 64, 0, kParts);
    const int c = (threadIdx.x & 7) * 8;
    float ws[8], xs[8], v[2][8];
    if (a.qx) load_part<FULL>(a.ws, n0 + c, a.N, ws);
    if (a.qw) load_part<FULL>(a.xs, m0 + c, a.M, xs);
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int m = m0 + (threadIdx.x >> 3) + 32 * k;
#pragma unroll
        for (int e = 0; e < 8; e++) v[k][e] = 0.0f;
        if (FULL || m < a.M) load_part<FULL>(static_cast<const T*>(a.dy) + m * a.ld, n0 + c, a.N, v[k]);
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int rr = (threadIdx.x >> 3) + 32 * k, m = m0 + rr;
        if constexpr (sizeof(T) == 2) {  // (the values as they were: their words)
#pragma unroll
            for (int e = 0; e < 8; e += 2) *reinterpret_cast<uint32_t*>(&tile[rr][c + e]) = pack16(v[k][e], v[k][e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) tile[rr][c + e] = v[k][e];
        }
        if (a.qx && (FULL || m < a.M)) {
            const float up = scale_up(a.rowmax[m]);
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; e++) p[e] = v[k][e] * ws[e] * up;
            store_parts(a.qx + m * rowx + part_at(cn, 0, kParts) + 2 * c, p);
        }
    }
    if (!a.qw) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int rr = (threadIdx.x >> 3) + 32 * k, n = n0 + rr;
        if (!FULL && n >= a.N) continue;
        const float up = scale_up(a.colmax[n]);
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if constexpr (sizeof(T) == 2) p[e] = bf16_bits_to_f32(tile[c + e][rr]) * xs[e] * up;
            else p[e] = tile[c + e][rr] * xs[e] * up;
        }
        store_parts(a.qw + n * roww + part_at(cm, 0, kParts) + 2 * c, p);
    }
}
// The sums of the blocks of 64 rows, in double and in a fixed order: 32 columns a workgroup, eight interleaved sums.
__device__ __forceinline__ void join_bias(const DyArgs& a, int block, double (&red)[8][32]) {
    const int l = threadIdx.x & 31, q = threadIdx.x >> 5, n = block * 32 + l, blocks = (a.M + 63) / 64;
    double s = 0.0;
    if (n < a.N) {
#pragma unroll 8
        for (int p = q; p < blocks; p += 8) s += a.part[static_cast<int64_t>(p) * a.N + n];
    }
    red[q][l] = s;
    __syncthreads();
    if (q == 0 && n < a.N) {
        s = 0.0;
#pragma unroll
        for (int k = 0; k < 8; k++) s += red[k][l];
        a.dbias[n] = static_cast<float>(s);
    }
}

// The first `bias` workgroups join dbias, the others lay out 64 x 64 of dy each.
template <class T>
__global__ __launch_bounds__(256) void lay_dy_kernel(DyArgs a, int bias) {
    __shared__ union {
        T tile[64][66];
        double red[8][32];
    } lds;
    if (static_cast<int>(blockIdx.x) < bias) return join_bias(a, blockIdx.x, lds.red);
    const int across = (a.N + 63) / 64, at = blockIdx.x - bias;
    const int cn = at % across, cm = at / across;
    if (a.wide && cm * 64 + 64 <= a.M && cn * 64 + 64 <= a.N) lay_dy<true>(a, cm, cn, lds.tile);
    else lay_dy<false>(a, cm, cn, lds.tile);
}

// Codes [R][C] (rows ld bytes apart, C a multiple of 16) to FP16, C rows of R in chunks of 64: 64 x 64 a
// workgroup (36 to 41 us for 32768 x 2048, 5.3 TB/s, a tenth of the
// cycles in LDS conflicts; 44 with the halves of a line on two dies).
struct Codes {
    const int8_t* codes;
    int64_t ld;
    int R, C;
    char* out;
    int blocks;
};
__device__ __forceinline__ void lay_codes(const Codes& a, int block, int8_t (&tile)[64][68]) {
    const int across = (a.C + 63) / 64;
    // (the halves of a line on one die, workgroups eight apart)
    if ((block | 15) < a.blocks) block = (block & ~15) | (block & 7) << 1 | (block >> 3 & 1);
    const int c0 = (block % across) * 64, cr = block / across, r0 = cr * 64;
    {
        const int rr = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;
        uv4 v = {};
        if (r0 + rr < a.R && c0 + c < a.C) v = load16(a.codes + (r0 + rr) * a.ld + c0 + c);
#pragma unroll
        for (int e = 0; e < 4; e++) *reinterpret_cast<uint32_t*>(&tile[rr][c + 4 * e]) = v[e];
    }
    __syncthreads();
    const int64_t row = part_at((a.R + 63) / 64, 0, 1);
    const int c = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int rr = (threadIdx.x >> 3) + 32 * k;
        if (c0 + rr >= a.C) continue;
        hv8 h;
#pragma unroll
        for (int e = 0; e < 8; e++) h[e] = static_cast<_Float16>(tile[c + e][rr]);
        *reinterpret_cast<hv8*>(a.out + (c0 + rr) * row + part_at(cr, 0, 1) + 2 * c) = h;
    }
}
// Both operands of codes, and zeros to what the maxima of dy go to.
__global__ __launch_bounds__(256) void lay_codes_kernel(Codes x, Codes w, uint32_t* clear, int64_t words) {
    __shared__ __align__(16) int8_t tile[64][68];
    const int b = blockIdx.x;
    if (b < x.blocks) return lay_codes(x, b, tile);
    if (b < x.blocks + w.blocks) return lay_codes(w, b - x.blocks, tile);
    const int64_t at = static_cast<int64_t>(b - x.blocks - w.blocks) * 1024 + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (at + 256 * k < words) clear[at + 256 * k] = 0;
}

// out[j][i] = scale_back(row j) times the sum over the parts of sums[p][j][i], in order; 4 columns a lane.
struct Join {
    const float* sums;
    int parts, I, out_dtype;
    int64_t n;  // I J
    const uint32_t* row;
    void* out;
    int blocks;
};
__device__ __forceinline__ void join(const Join& a, int block) {
    const int64_t at = (static_cast<int64_t>(block) * 256 + threadIdx.x) * 4;
    if (at >= a.n) return;
    double s[4] = {};
    for (int p = 0; p < a.parts; p++) {
        const fv4 v = *reinterpret_cast<const fv4*>(a.sums + p * a.n + at);
#pragma unroll
        for (int e = 0; e < 4; e++) s[e] += v[e];
    }
    const float k = scale_back(a.row[at / a.I]);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = static_cast<float>(s[e]) * k;
    if (a.out_dtype == LA_BF16) *reinterpret_cast<uv2*>(static_cast<uint16_t*>(a.out) + at) = uv2{pack16(v[0], v[1]), pack16(v[2], v[3])};
    else *reinterpret_cast<fv4*>(static_cast<float*>(a.out) + at) = fv4{v[0], v[1], v[2], v[3]};
}
__global__ __launch_bounds__(256) void join_kernel(Join x, Join w) {
    const int b = blockIdx.x;
    if (b < x.blocks) join(x, b);
    else join(w, b - x.blocks);
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// What the workspace holds, in this order.
struct Layout {
    size_t rowmax, colmax, part, qx, qw, pw, px, sums_x, sums_w, end;  // offsets; pw: w's codes, px: x's
    Cut dx, dw;            // the two products,
    bool pair;             // which may share a launch
};
Layout layout(const la_linear_config& c) {
    Layout l;
    const size_t M = c.M, N = c.N, K = c.K, mc = (M + 63) / 64, nc = (N + 63) / 64;
    size_t at = 0;
    auto take = [&](size_t n) { const size_t p = at; at += up256(n); return p; };
    l.rowmax = take(4 * M), l.colmax = take(4 * N), l.part = take(4 * mc * N);
    l.qx = take(M * nc * 128 * kParts), l.qw = take(N * mc * 128 * kParts);
    l.pw = take(K * nc * 128), l.px = take(K * mc * 128);
    const GradientCuts cuts = cut_gradients(c.M, c.N, c.K);
    l.dx = cuts.dx, l.dw = cuts.dw, l.pair = cuts.pair;
    l.sums_x = take(l.dx.parts > 1 ? l.dx.parts * M * K * 4 : 0);
    l.sums_w = take(l.dw.parts > 1 ? l.dw.parts * N * K * 4 : 0);
    l.end = at;
    return l;
}

// Cuts a product's sum into parts, which go to `sums` and are left to `join`.
void cut(GemmArgs& g, const Cut& cut, float* sums, Join& join) {
    g.parts = cut.parts;
    g.part_steps = (gemm_steps(g.kbytes, g.shift) + cut.parts - 1) / cut.parts;
    if (cut.parts == 1) return;
    const int64_t n = static_cast<int64_t>(g.I) * g.J;
    join = {sums, cut.parts, g.I, g.out_dtype, n, static_cast<const uint32_t*>(g.row), g.out, static_cast<int>((n / 4 + 255) / 256)};
    g.row = nullptr, g.out = sums, g.out_dtype = LA_F32;
}

// Without tokens or channels every sum is empty: zeros, and no operand is looked at (the call may have none).
bool no_sums(const la_linear_config& c) { return c.M == 0 || c.N == 0; }

}  // namespace

size_t linear_bwd_workspace(const la_linear_config& c) { return no_sums(c) ? 0 : layout(c).end; }

hipError_t launch_linear_bwd(const la_linear_config& c, const LinearArgs& a, hipStream_t s) {
    if (no_sums(c)) {
        for (const hipError_t e : {launch_zero_rows(a.dx, c.x_dtype, c.M, c.K, c.K, s), launch_zero_rows(a.dw, c.dw_dtype, c.N, c.K, c.K, s),
                                   launch_zero_rows(a.dbias, LA_F32, 1, c.N, c.N, s)})
            if (e != hipSuccess) return e;
        return hipSuccess;
    }
    const Layout l = layout(c);
    const int es = c.out_dtype == LA_BF16 ? 2 : 4;
    DyArgs d{};
    d.dy = a.dy, d.xs = a.xs, d.ws = a.ws, d.M = c.M, d.N = c.N, d.ld = c.ld_y ? c.ld_y : c.N;
    d.wide = d.ld * es % 16 == 0;
    d.rowmax = a.dx ? reinterpret_cast<uint32_t*>(a.work + l.rowmax) : nullptr;
    d.colmax = a.dw ? reinterpret_cast<uint32_t*>(a.work + l.colmax) : nullptr;
    d.part = a.dbias ? reinterpret_cast<float*>(a.work + l.part) : nullptr, d.dbias = a.dbias;
    d.qx = a.dx ? a.work + l.qx : nullptr, d.qw = a.dw ? a.work + l.qw : nullptr;
    const int64_t words = static_cast<int64_t>((l.part - l.rowmax) / 4);
    const int64_t mc = (c.M + 63) / 64, nc = (c.N + 63) / 64, kc = (c.K + 63) / 64;
    const Codes x{a.x, c.ld_x ? c.ld_x : c.K, c.M, c.K, a.work + l.px, a.dw ? static_cast<int>(mc * kc) : 0};
    const Codes w{a.w, c.K, c.N, c.K, a.work + l.pw, a.dx ? static_cast<int>(nc * kc) : 0};
    const int64_t first = x.blocks + w.blocks + (words + 1023) / 1024;
    lay_codes_kernel<<<static_cast<unsigned>(first), 256, 0, s>>>(x, w, reinterpret_cast<uint32_t*>(a.work + l.rowmax), words);
    const int64_t stats = mc * ((c.N + 255) / 256), bias = a.dbias ? (c.N + 31) / 32 : 0, lay = bias + (a.dx || a.dw ? mc * nc : 0);
    if (es == 2) {
        stats_kernel<uint16_t><<<static_cast<unsigned>(stats), 256, 0, s>>>(d);
        lay_dy_kernel<uint16_t><<<static_cast<unsigned>(lay), 256, 0, s>>>(d, static_cast<int>(bias));
    } else {
        stats_kernel<float><<<static_cast<unsigned>(stats), 256, 0, s>>>(d);
        lay_dy_kernel<float><<<static_cast<unsigned>(lay), 256, 0, s>>>(d, static_cast<int>(bias));
    }
    if (hipError_t e = hipGetLastError()) return e;
    const bool dx = a.dx, dw = a.dw;
    GemmArgs gx, gw;
    Join jx{}, jw{};
    if (dx) {
        gx.P = a.work + l.pw, gx.ldP = nc * 128, gx.I = c.K, gx.kbytes = static_cast<int>(nc * 128);
        gx.Q = d.qx, gx.ldQ = nc * 128 * kParts, gx.J = c.M, gx.shift = kShift;
        gx.row = d.rowmax, gx.out = a.dx, gx.out_dtype = c.x_dtype, gx.ldo = c.K, gx.wide = 1;
        cut(gx, l.dx, reinterpret_cast<float*>(a.work + l.sums_x), jx);
    }
    if (dw) {
        gw.P = a.work + l.px, gw.ldP = mc * 128, gw.I = c.K, gw.kbytes = static_cast<int>(mc * 128);
        gw.Q = d.qw, gw.ldQ = mc * 128 * kParts, gw.J = c.N, gw.shift = kShift;
        gw.row = d.colmax, gw.out = a.dw, gw.out_dtype = c.dw_dtype, gw.ldo = c.K, gw.wide = 1;
        cut(gw, l.dw, reinterpret_cast<float*>(a.work + l.sums_w), jw);
    }
    if (dx && dw && l.pair) {
        if (hipError_t e = launch_pair<_Float16, true>(gx, gw, l.dx.tiling, s)) return e;
    } else {
        if (dx)
            if (hipError_t e = launch_gemm<_Float16, true>(gx, l.dx.tiling, s)) return e;
        if (dw)
            if (hipError_t e = launch_gemm<_Float16, true>(gw, l.dw.tiling, s)) return e;
    }
    if (jx.blocks + jw.blocks > 0) join_kernel<<<static_cast<unsigned>(jx.blocks + jw.blocks), 256, 0, s>>>(jx, jw);
    return hipGetLastError();
}

}  // namespace la
