// Selective scan forward: a workgroup walks the 64-token chunks of one sequence for 64 or 128
// value columns, the states in its accumulators.
//
// Only the states' update is serial.  Eight waves, two roles, two barriers a step; at step i
//   waves 0..3   bring chunk i into LDS | form its M and the decays of chunk i + 1
//   waves 4..7   (16 or 32 columns each) form M x and W x of chunk i - 1 | add the state's part,
//                write the output and update the state
// with two LDS buffers and the loads of chunk i + 2 issued at step i.  M and the state enter the
// products as two bf16 parts (2^-17 of a value, for a bf16 result), W x as three (exact; two
// cost a tenth of the time less, but the final states were then further from their 64-bit values
// than FP32 arithmetic's).  bf16 results lie 1.0e-4 from those of FP32 arithmetic, most of it from D x,
// where D sits on M's diagonal, and as near to their 64-bit values (1.66e-3); D x added by itself
// took that to 2.7e-5 and to the same 1.66e-3, for 3 to 7% more time.  LDS and the chain of reads, products and operand splits of waves 4..7 bound it, not
// memory: with d_k = 128 a chunk takes 2.8 us for 64 columns, 4.7 us for 128.  8 sequences of
// 4096 tokens, 16 heads, d_v = 128: 182 us by the clock, 196 by the profiler; 64 packed sequences,
// 40686 tokens in all: 245 to 262 us and 277.
// Every wave doing every part in turn took 5.3 us a chunk of 64 columns; sixteen waves in the
// same roles 5% more, and c's rows loaded from memory by waves 4..7 themselves 60% more than this.
//
// Few heads and long sequences: the walk is cut into segments that run side by side.  A first
// pass forms each segment's own contribution to the state from zero, a small kernel joins them
// (S_in of every segment), and the full walk starts every segment from its S_in (32768 tokens,
// 32 heads of d_v = 64: 80 + 8 + 168 us by the profiler, 214 to 219 us by the clock).
#include "la_scan.hpp"

namespace la {
namespace {

// CT: 64-column tiles a workgroup; HEADS: heads that they belong to (1, or CT heads of one tile each).
template <class T, int N, int CT, int HEADS, bool FULL>
struct FwdBuf {
    T b[kQ * lds_row<T>(N)];
    T c[FULL ? kQ * lds_row<T>(N) : 8];
    T x[kQ * (CT == 2 ? lds_row<T>(128) : lds_row64<T>())];
};
template <class T, int N, int CT, int HEADS, bool FULL, int NB>
struct FwdLds {
    FwdBuf<T, N, CT, HEADS, FULL> buf[NB];
    T m[FULL ? HEADS : 1][FULL ? Mat<T>::template parts<2> : 1][FULL ? kQ * lds_row64<T>() : 8];
    Decay d[3][HEADS];  // formed a chunk earlier
};
// Two buffers where they fit (160 KB; not FP32 with d_k = 128: the roles then take turns).
template <class T, int N, int CT, int HEADS, bool FULL>
constexpr int kBufs = sizeof(FwdLds<T, N, CT, HEADS, FULL, 2>) <= 160 * 1024 ? 2 : 1;
template <class T, int N, int CT, int HEADS, bool FULL>
using FwdShared = FwdLds<T, N, CT, HEADS, FULL, kBufs<T, N, CT, HEADS, FULL>>;

// FULL: outputs and S_T, from the segment's S_in (or S0).  Otherwise the segment's state from
// zero into `local` and its decay into `decay`.
template <class T, int N, int CT, int HEADS, bool FULL>
__global__ __launch_bounds__(512) void scan_fwd_kernel(ScanP p, const float* S0, const float* Sin, void* y, float* ST,
                                                       float* local, float* decay, int nseg, int segs) {
    using MT = Mat<T>;
    constexpr int P2 = MT::template parts<2>, P3 = MT::template parts<3>;
    constexpr int COLS = kPT * CT;
    constexpr int RB = lds_row<T>(N), RX = CT == 2 ? lds_row<T>(128) : lds_row64<T>(), RM = lds_row64<T>();
    constexpr int KS = N / 32;  // contraction steps over the state's rows
    constexpr int NB = kBufs<T, N, CT, HEADS, FULL>;
    using Buf = FwdBuf<T, N, CT, HEADS, FULL>;
    extern __shared__ __align__(16) char raw_lds[];
    FwdShared<T, N, CT, HEADS, FULL>& shared = *reinterpret_cast<FwdShared<T, N, CT, HEADS, FULL>*>(raw_lds);
    Buf* const bufs = shared.buf;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lm = lane & 15, g = lane >> 4;

    const int tiles = HEADS == 1 ? p.dv / COLS : 1;
    uint32_t u = die_unit(blockIdx.x, gridDim.x);
    const int tile = take(u, tiles), h = take(u, p.H / HEADS) * HEADS, seg = take(u, segs);  // segs: segments of this launch
    const int bi = static_cast<int>(u);
    uint32_t hu = static_cast<uint32_t>(h);
    take(hu, p.H / p.G);
    const int grp = static_cast<int>(hu);

    const SeqRange sr = seq_range(p, bi);
    const int nch = (sr.len + kQ - 1) / kQ;
    const int cps = (nch + nseg - 1) / nseg;
    const int c0 = seg * cps;
    const int c1 = c0 + cps < nch ? c0 + cps : nch;
    if (c0 >= nch && !(nch == 0 && seg == 0)) return;
    float A[HEADS], Dh[HEADS], bias[HEADS];
#pragma unroll
    for (int q = 0; q < HEADS; q++) {
        A[q] = p.A ? p.A[h + q] : 0.0f;  // (no tokens: A may be missing)
        Dh[q] = FULL && p.D ? p.D[h + q] : 0.0f;
        bias[q] = p.bias ? p.bias[h + q] : 0.0f;
    }

    if (FULL) {  // the tiles above the diagonal that the products below read stay zero
        for (int i = threadIdx.x; i < HEADS * P2 * kQ * RM; i += 512) (&shared.m[0][0][0])[i] = T{};
        __syncthreads();
    }

    if (wave < 4) {
        // ------------------------------------------------------------ chunks into LDS, and M
        const T* xg = static_cast<const T*>(p.x) + static_cast<int64_t>(h) * p.dv + tile * COLS;
        const T* bg = static_cast<const T*>(p.b) + static_cast<int64_t>(grp) * p.dk;
        const T* cg = static_cast<const T*>(p.c) + static_cast<int64_t>(grp) * p.dk;
        struct None {};
        struct Ahead {
            Tile<T, N, 256> b;
            std::conditional_t<FULL, Tile<T, N, 256>, None> c;
            Tile<T, COLS, 256> x;
            DtAhead raw[HEADS];
        };
        // two chunks ahead (FP32 tiles are twice the registers: one)
        constexpr int AH = sizeof(T) == 2 && NB == 2 ? 2 : 1;
        Ahead even, odd;
        auto fetch = [&](int ch, Ahead& r) {
            if (ch >= c1) return;
            const int64_t row0 = sr.begin + static_cast<int64_t>(ch) * kQ;
            const int live = sr.len - ch * kQ;
            r.b.load(bg + row0 * p.ld_b, p.ld_b, live, p.dk);
            if constexpr (FULL) r.c.load(cg + row0 * p.ld_c, p.ld_c, live, p.dk);
            r.x.load(xg + row0 * p.ld_x, p.ld_x, live, COLS);
            if (wave == 3)
#pragma unroll
                for (int q = 0; q < HEADS; q++) r.raw[q].fetch(p, row0, h + q, lane, live);
        };
        double cum_seg[HEADS] = {};
        auto decays_of = [&](int ch, const Ahead& r) {  // by one wave
#pragma unroll
            for (int q = 0; q < HEADS; q++)
                cum_seg[q] += make_decay(shared.d[(ch - c0) % 3][q], r.raw[q].value(p) + bias[q], p.softplus, sr.len - ch * kQ, A[q]);
        };
        auto stage = [&](Buf& lds, const Ahead& r) {
            r.b.store(lds.b, RB);
            if constexpr (FULL) r.c.store(lds.c, RB);
            r.x.store(lds.x, RX);
        };
        // M^T tile (ti, si): rows s, columns t; lane: t, four consecutive s.  D goes onto the diagonal.
        auto pair = [&](Buf& lds, const Decay* ds, int ti, int si) {
            const int ln = opaque(lane), lm = ln & 15, g = ln >> 4;
            const int t = 16 * ti + lm, s0 = 16 * si + 4 * g;
            typename MT::Frag bf[KS], cf[KS];
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
                cf[ks] = MT::row8(lds.c + t * RB + 32 * ks + 8 * g);
                bf[ks] = MT::row8(lds.b + (16 * si + lm) * RB + 32 * ks + 8 * g);
            }
            float thi[HEADS], tlo[HEADS];
            f4 shi[HEADS], slo[HEADS], sdl[HEADS];
#pragma unroll
            for (int q = 0; q < HEADS; q++) {
                thi[q] = ds[q].hi[t], tlo[q] = ds[q].lo[t];
                shi[q] = *reinterpret_cast<const f4*>(ds[q].hi + s0);
                slo[q] = *reinterpret_cast<const f4*>(ds[q].lo + s0);
                sdl[q] = *reinterpret_cast<const f4*>(ds[q].delta + s0);
            }
            __builtin_amdgcn_sched_barrier(0);
            f4 acc = {};
#pragma unroll
            for (int ks = 0; ks < KS; ks++) acc = MT::mma(bf[ks], cf[ks], acc);
#pragma unroll
            for (int q = 0; q < HEADS; q++) {
                float m[4];
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    m[r] = acc[r] * (pair_decay(thi[q], tlo[q], shi[q][r], slo[q][r]) * sdl[q][r]);
                    if (si == ti) m[r] = s0 + r < t ? m[r] : s0 + r == t ? m[r] + Dh[q] : 0.0f;
                }
                MT::template put4<P2>(&shared.m[q][0][t * RM + s0], kQ * RM, m);
            }
        };
        auto pairs = [&](Buf& lds, const Decay* d) {  // the ten tiles; the wave with one also forms the decays
            if constexpr (FULL) {
                if (wave < 2) {
                    for (int si = 0; si < 3; si++) pair(lds, d, 3 - wave, si);
                } else if (wave == 2) {
                    for (int si = 0; si < 2; si++) pair(lds, d, 1, si);
                    pair(lds, d, 3, 3);
                } else {
                    pair(lds, d, 0, 0);
                }
            }
        };
        fetch(c0, even);
        if constexpr (AH == 2) fetch(c0 + 1, odd);
        if constexpr (NB == 2) {
            // r holds chunk ch, next chunk ch + 1 (one register set: after its refill)
            auto step = [&](int ch, Buf& lds, Ahead& r, Ahead& next) {
                if (ch < c1) {
                    stage(lds, r);
                    if (wave == 3 && (!FULL || ch == c0)) decays_of(ch, r);
                    fetch(ch + AH, r);
                }
                __syncthreads();
                if constexpr (FULL) {
                    if (ch < c1) pairs(lds, shared.d[(ch - c0) % 3]);
                    if (wave == 3 && ch + 1 < c1) decays_of(ch + 1, next);
                    __syncthreads();
                }
            };
            for (int ch = c0; ch <= c1; ch += 2) {  // chunk c1: the other role's last
                if constexpr (AH == 2) {
                    step(ch, bufs[0], even, odd);
                    if (ch + 1 <= c1) step(ch + 1, bufs[1], odd, even);
                } else {
                    step(ch, bufs[0], even, even);
                    if (ch + 1 <= c1) step(ch + 1, bufs[1], even, even);
                }
            }
        } else {
            for (int ch = c0; ch < c1; ch++) {
                stage(bufs[0], even);
                if (wave == 3) decays_of(ch, even);
                fetch(ch + 1, even);
                __syncthreads();
                if (FULL) {
                    pairs(bufs[0], shared.d[(ch - c0) % 3]);
                    __syncthreads();
                }
                __syncthreads();
            }
        }
        if (!FULL && threadIdx.x == 192 && tile == 0)
#pragma unroll
            for (int q = 0; q < HEADS; q++)
                decay[(static_cast<size_t>(bi) * nseg + seg) * p.H + h + q] = static_cast<float>(exp2(cum_seg[q]));
        return;
    }

    // ---------------------------------------------------------------- outputs and the state
    const int w0 = 16 * CT * (wave - 4);  // this wave's columns of the tile, 16 at a time
    const int hh = HEADS == 1 ? 0 : (wave - 4) / 2;  // (two heads: 32 columns are half of one's)
    const int hw = h + hh;
    f4 S[CT][N / 16];                     // a lane: column w0 + 16 c + lm
    const size_t unit = (static_cast<size_t>(bi) * p.H + hw) * p.dk * p.dv;
    const int pcol = tile * COLS + w0 - kPT * hh + lm;
    const float* init = nullptr;
    if (FULL) init = nseg > 1 && nch > 0 ? Sin + ((static_cast<size_t>(bi) * nseg + seg) * p.H + hw) * p.dk * p.dv
                                         : (S0 ? S0 + unit : nullptr);
#pragma unroll
    for (int c = 0; c < CT; c++)
#pragma unroll
        for (int i = 0; i < N / 16; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int n = state_n(i, 4 * g + r);
                S[c][i][r] = init && n < p.dk ? init[static_cast<size_t>(n) * p.dv + pcol + 16 * c] : 0.0f;
            }
    // LDS reads are issued together ahead of the products that take them (the fences keep the
    // compiler from sinking each to its use, where its whole latency would be waited for), and
    // products on one accumulator are kept four apart.
    //
    // What needs no state: W x, and M x as y^T (rows: columns w0 + 16 c + 4 g + r of x; column: t).
    auto stateless = [&](const Buf& lds, const Decay& d, f4 (&acc)[CT][4], typename MT::Frag (&wx)[CT][2][P3]) {
        const int ln = opaque(lane), lm = ln & 15, g = ln >> 4;
        typename MT::Frag xT[CT][2], mf[2][P2][4];  // x^T: column w0 + 16 c + lm
        float wt[2][8];
#pragma unroll
        for (int k = 0; k < 2; k++) {
#pragma unroll
            for (int c = 0; c < CT; c++) xT[c][k] = MT::col8(lds.x, RX, 32 * k, w0 + 16 * c, ln);
            get8(d.w + 32 * k + 8 * g, wt[k]);
        }
        if constexpr (FULL) {
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
#pragma unroll
                for (int k = 0; k < P2; k++)
#pragma unroll
                    for (int i = 2 * ks; i < 4; i++) mf[ks][k][i] = MT::row8(&shared.m[hh][k][(16 * i + lm) * RM + 32 * ks + 8 * g]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < CT; c++)
#pragma unroll
                for (int i = 0; i < 4; i++) acc[c][i] = f4{};
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
#pragma unroll
                for (int k = 0; k < P2; k++)
#pragma unroll
                    for (int c = 0; c < CT; c++)
#pragma unroll
                        for (int i = 2 * ks; i < 4; i++) acc[c][i] = MT::mma(xT[c][ks], mf[ks][k][i], acc[c][i]);
        }
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int k = 0; k < 2; k++) {
                float v[8];
                MT::widen8(xT[c][k], v);
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] *= wt[k][j];
                MT::template split<P3>(v, wx[c][k]);
            }
    };
    const int es = p.out_dtype == LA_BF16 ? 2 : 4;
    const int64_t ld_y = static_cast<int64_t>(p.H) * p.dv;
    // contraction steps whose c rows are read together (two tiles leave registers for one)
    constexpr int AHEAD = sizeof(T) == 2 && CT == 1 ? KS : 1;
    auto output = [&](int ch, const Buf& lds, const Decay& d, const f4 (&acc)[CT][4]) {
        const int ln = opaque(lane), lm = ln & 15, g = ln >> 4;
        f4 y4[CT][4] = {};
        float head[4];
#pragma unroll
        for (int i = 0; i < 4; i++) head[i] = d.head[16 * i + lm];
#pragma unroll
        for (int k0 = 0; k0 < KS; k0 += AHEAD) {
            typename MT::Frag cf[AHEAD][4];
#pragma unroll
            for (int ks = 0; ks < AHEAD; ks++)
#pragma unroll
                for (int i = 0; i < 4; i++) cf[ks][i] = MT::row8(lds.c + (16 * i + lm) * RB + 32 * (k0 + ks) + 8 * g);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ks = 0; ks < AHEAD; ks++)
#pragma unroll
                for (int c = 0; c < CT; c++) {
                    const f4 &a = S[c][2 * (k0 + ks)], &b = S[c][2 * (k0 + ks) + 1];
                    typename MT::Frag Sp[P2];
                    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                    MT::template split<P2>(v, Sp);
#pragma unroll
                    for (int k = 0; k < P2; k++)
#pragma unroll
                        for (int i = 0; i < 4; i++) y4[c][i] = MT::mma(Sp[k], cf[ks][i], y4[c][i]);
                }
        }
        // rows behind the sequence lie behind the buffer's end
        const int live = sr.len - ch * kQ < kQ ? sr.len - ch * kQ : kQ;
        char* row0 = static_cast<char*>(y) + ((sr.begin + ch * static_cast<int64_t>(kQ)) * ld_y + static_cast<int64_t>(h) * p.dv + tile * COLS) * es;
        const __amdgpu_buffer_rsrc_t ry = make_rsrc(row0, static_cast<size_t>(live) * ld_y * es);
#pragma unroll
        for (int c = 0; c < CT; c++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                f4 v;
#pragma unroll
                for (int r = 0; r < 4; r++) v[r] = __builtin_fmaf(y4[c][i][r], head[i], acc[c][i][r]);
                const int off = ((16 * i + lm) * static_cast<int>(ld_y) + w0 + 16 * c + 4 * g) * es;
                if (es == 2)
                    __builtin_amdgcn_raw_buffer_store_b64(uv2{pack16(v[0], v[1]), pack16(v[2], v[3])}, ry, off, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uv4, v), ry, off, 0, 0);
            }
    };
    auto update = [&](const Buf& lds, const Decay& d, const typename MT::Frag (&wx)[CT][2][P3]) {  // S = total S + B^T (W x)
        const int ln = opaque(lane);
        const float total = d.total[0];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            typename MT::Frag bf[N / 16];
#pragma unroll
            for (int i = 0; i < N / 16; i++) bf[i] = MT::col8_state(lds.b, RB, 32 * k, i, ln);
            __builtin_amdgcn_sched_barrier(0);
            if (k == 0) {
#pragma unroll
                for (int c = 0; c < CT; c++)
#pragma unroll
                    for (int i = 0; i < N / 16; i++) S[c][i] *= total;
            }
#pragma unroll
            for (int q = 0; q < P3; q++)
#pragma unroll
                for (int c = 0; c < CT; c++)
#pragma unroll
                    for (int i = 0; i < N / 16; i++) S[c][i] = MT::mma(bf[i], wx[c][k][q], S[c][i]);
        }
    };
    if constexpr (NB == 2) {
        auto step = [&](int ch, const Buf& lds) {  // beside the staging of chunk ch + 1 and its M
            const Decay& d = shared.d[(ch - c0 + 3) % 3][hh];
            typename MT::Frag wx[CT][2][P3];
            f4 acc[CT][4];
            if (ch >= c0) stateless(lds, d, acc, wx);
            if constexpr (FULL) {
                __syncthreads();
                if (ch >= c0) output(ch, lds, d, acc);
            }
            if (ch >= c0) update(lds, d, wx);
            __syncthreads();
        };
        for (int ch = c0; ch <= c1; ch += 2) {
            step(ch - 1, bufs[1]);
            if (ch + 1 <= c1) step(ch, bufs[0]);
        }
    } else {
        for (int ch = c0; ch < c1; ch++) {
            const Decay& d = shared.d[(ch - c0) % 3][hh];
            typename MT::Frag wx[CT][2][P3];
            f4 acc[CT][4];
            __syncthreads();
            if (FULL) __syncthreads();
            stateless(bufs[0], d, acc, wx);
            if (FULL) output(ch, bufs[0], d, acc);
            update(bufs[0], d, wx);
            __syncthreads();
        }
    }
    float* out = nullptr;
    if (FULL) out = c1 == nch && ST ? ST + unit : nullptr;
    else out = local + ((static_cast<size_t>(bi) * nseg + seg) * p.H + hw) * p.dk * p.dv;
    if (!out) return;
#pragma unroll
    for (int c = 0; c < CT; c++)
#pragma unroll
        for (int i = 0; i < N / 16; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int n = state_n(i, 4 * g + r);
                if (n < p.dk) out[static_cast<size_t>(n) * p.dv + pcol + 16 * c] = S[c][i][r];
            }
}

// The state entering every segment from the segments' own states, in place.
__global__ __launch_bounds__(256) void scan_join_kernel(ScanP p, const float* S0, float* local, const float* decay, int nseg) {
    const int per = p.dk * p.dv / 4;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<int64_t>(p.B) * p.H * per) return;
    const int e = static_cast<int>(i % per);
    const int64_t bh = i / per;
    const int h = static_cast<int>(bh % p.H), bi = static_cast<int>(bh / p.H);
    const int nch = (seq_range(p, bi).len + kQ - 1) / kQ;
    const int cps = (nch + nseg - 1) / nseg;
    fv4 S = {};
    if (S0) S = reinterpret_cast<const fv4*>(S0)[bh * per + e];
    const int used = cps > 0 ? (nch + cps - 1) / cps : 0;  // the last segment's own state is not formed
    for (int s0 = 0; s0 < used; s0 += 8) {                 // eight segments' loads in flight
        fv4 own[8];
        float dec[8];
        fv4* l[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int s = s0 + j < used ? s0 + j : used - 1;
            const size_t at = (static_cast<size_t>(bi) * nseg + s) * p.H + h;
            l[j] = reinterpret_cast<fv4*>(local) + at * per + e;
            const bool more = s + 1 < used;
            own[j] = more ? *l[j] : fv4{};
            dec[j] = more ? decay[at] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (s0 + j >= used) break;
            *l[j] = S;
            S = S * dec[j] + own[j];
        }
    }
}

// Columns a workgroup and segments of a sequence.
struct Walk {
    int tiles, heads;  // 64-column tiles, and the heads that they belong to
    int nseg;
};
// Segments: one while the heads alone fill the chip, else enough for that: the first pass costs
// about half a full walk, so that a cut of one-tile walks pays from three segments on.  A segment
// has two chunks at least, or three of bf16 where there are few (whose walk costs little more
// than the join: 1024 tokens, 16 heads of 128: 35-36 us with 3 or 4, 37 with 2; 700 tokens, 4
// heads: 29 with 3, 31 with 2, 36 with 4; but 2048 tokens: 45 with 2, 48 with 4, and 1000 FP32
// tokens, 8 heads: 31 against 39).
//
// One tile a workgroup, or two (a head's 128 columns, or two heads of one group), where b, c and
// their products serve both, but half as many workgroups walk.  Two pay where they still fill
// the chip (2048 tokens, 16 sequences of 16 heads, d_v = 128: 177 -> 135 us; 40686 packed tokens:
// 337 -> 261) or where the walk is cut into segments either way (32768 tokens, 16 heads of 128:
// 243 -> 206 us; 32 of 64: 244 -> 216); not for 256 tiles, where one a workgroup fills the chip
// without a cut (4096 tokens, 8 sequences of 16 heads: 166 against 202 us in two segments).
Walk walk_of(const la_scan_config& c) {
    const int64_t groups = static_cast<int64_t>(c.B) * c.H * (c.d_v / kPT);
    const int64_t chunks = (c.T + kQ - 1) / kQ;
    if (groups == 0) return {1, 1, 1};
    const int least = c.x_dtype == LA_F32 || chunks >= 32 ? 2 : 3;
    auto cut = [&](int64_t most) { return most < chunks / least ? most : chunks / least; };
    int64_t n = cut(512 / groups);
    if (n < 3) n = 1;
    const int heads = c.d_v % 128 == 0 ? 1 : c.d_v == 64 && (c.H / c.G) % 2 == 0 ? 2 : 0;
    if (c.x_dtype == LA_BF16 && heads && (groups >= 512 || (n > 1 && groups * n >= 256))) {
        n = cut(256 / (groups / 2));
        return {2, heads, n < 2 ? 1 : static_cast<int>(n)};
    }
    return {1, 1, static_cast<int>(n)};
}

size_t local_bytes(const la_scan_config& c, int nseg) {
    return static_cast<size_t>(c.B) * nseg * c.H * c.d_k * c.d_v * sizeof(float);
}

template <class T, int N, int CT, int HEADS>
hipError_t launch_walk(const la_scan_config& c, const ScanArgs& a, int nseg, hipStream_t s) {
    const ScanP p = scan_params(c, a);
    const int64_t groups = static_cast<int64_t>(c.B) * c.H * (c.d_v / kPT) / CT;
    float* local = reinterpret_cast<float*>(a.ws);
    float* decay = reinterpret_cast<float*>(a.ws + (nseg > 1 ? local_bytes(c, nseg) : 0));
    auto allow = [](auto& kernel, size_t bytes) {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(bytes));
    };
    hipError_t e;
    if (nseg > 1) {
        constexpr size_t bytes = sizeof(FwdShared<T, N, CT, HEADS, false>);
        e = allow(scan_fwd_kernel<T, N, CT, HEADS, false>, bytes);
        if (e != hipSuccess) return e;
        scan_fwd_kernel<T, N, CT, HEADS, false><<<dim3(static_cast<unsigned>(groups * (nseg - 1))), 512, bytes, s>>>(
            p, nullptr, nullptr, nullptr, nullptr, local, decay, nseg, nseg - 1);
        const int64_t items = static_cast<int64_t>(c.B) * c.H * (c.d_k * c.d_v / 4);
        scan_join_kernel<<<dim3(static_cast<unsigned>((items + 255) / 256)), 256, 0, s>>>(p, a.S0, local, decay, nseg);
    }
    constexpr size_t bytes = sizeof(FwdShared<T, N, CT, HEADS, true>);
    e = allow(scan_fwd_kernel<T, N, CT, HEADS, true>, bytes);
    if (e != hipSuccess) return e;
    scan_fwd_kernel<T, N, CT, HEADS, true><<<dim3(static_cast<unsigned>(groups * nseg)), 512, bytes, s>>>(
        p, a.S0, local, a.y, a.ST, nullptr, nullptr, nseg, nseg);
    return hipGetLastError();
}

template <class T, int N>
hipError_t launch(const la_scan_config& c, const ScanArgs& a, hipStream_t s) {
    const Walk w = walk_of(c);
    if constexpr (sizeof(T) == 2) {
        if (w.tiles == 2) return w.heads == 2 ? launch_walk<T, N, 2, 2>(c, a, w.nseg, s) : launch_walk<T, N, 2, 1>(c, a, w.nseg, s);
    }
    return launch_walk<T, N, 1, 1>(c, a, w.nseg, s);
}

}  // namespace

size_t scan_fwd_workspace(const la_scan_config& c) {
    const int nseg = walk_of(c).nseg;
    return nseg > 1 ? local_bytes(c, nseg) + static_cast<size_t>(c.B) * nseg * c.H * sizeof(float) : 0;
}

hipError_t launch_scan_fwd(const la_scan_config& c, const ScanArgs& a, hipStream_t s) {
    if (c.x_dtype == LA_BF16) {
        switch (c.d_k) {
            case 128: return launch<uint16_t, 128>(c, a, s);
            case 64: return launch<uint16_t, 64>(c, a, s);
            default: return launch<uint16_t, 32>(c, a, s);
        }
    }
    switch (c.d_k) {
        case 128: return launch<float, 128>(c, a, s);
        case 64: return launch<float, 64>(c, a, s);
        default: return launch<float, 32>(c, a, s);
    }
}

}  // namespace la
