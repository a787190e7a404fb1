// Selective scan backward.
//
// Two walks leave, for every 64-token chunk, the state S entering it and the gradient dS of the
// state leaving it (S_end) in the workspace; the gradients of a chunk then need nothing outside
// it and all chunks run side by side.  With dM = dY X^T, P = G o L o dM and dG = L o Delta o dM:
//     dX = M^T dY + diag(W) (B dS) + D dY          dS entering = exp(cum_end) dS + C^T diag(exp cum) dY
//     dC = sum over heads of dG B + diag(exp cum) (dY S^T)
//     dB = sum over heads of dG^T C + diag(W) (X dS^T)
//     c_s = column sums of P + tail_s b_s^T dS x_s         (dDelta_s but for P_ss and the decay's part)
//     r_t = row sums of P Delta + exp(cum_t) c_t^T S dy_t
// cum_t enters the chunk's results as exp(cum_t) on the rows and exp(-cum_s) on the columns (not P's
// diagonal, which both sums leave out: its decay is 1, and its rounding would not cancel), so its
// gradient is r_t - Delta_t c_t, plus for the last token exp(cum_end) <S, dS> + sum_s Delta_s
// (c_s's part from dS); a log decay's gradient is the suffix sum of those (in double: the terms
// cancel), and dDelta, dA follow from it.
//
// 8 sequences of 4096 tokens, 16 heads, 128 x 128, bf16 (the profiler's medians): decays 7 us, walks
// 338 us (0.35 GB read, 1.09 GB written, 4.3 TB/s), gradients 462 us (1.38 GB read, 0.17 GB written,
// 3.3 TB/s), rates 9 us, sums 5 us; one bf16 part for M and dG: 423 us.  64 packed sequences, 40686
// tokens in all: 1141 us.
// The FP32 states are 2.1 of those 2.8 GB.  Past the caches their stores and loads cost 4 to 6%.
#include "la_scan.hpp"

namespace la {
namespace {

// Chunk slots: dense, b nch + ch; packed, b + begin_b / 64 + ch (disjoint for any packing).
__device__ __forceinline__ int64_t slot_of(const ScanP& p, int b, int64_t begin, int ch) {
    if (!p.cu) return static_cast<int64_t>(b) * ((p.T + kQ - 1) / kQ) + ch;
    return b + begin / kQ + ch;
}
int64_t slot_count(const la_scan_config& c, bool packed) {
    return packed ? static_cast<int64_t>(c.B) + c.T / kQ + 1 : static_cast<int64_t>(c.B) * ((c.T + kQ - 1) / kQ);
}
// The chunk of a slot; a packing leaves some slots without one.
struct ChunkAt {
    int b, ch;
    SeqRange sr;
    bool used;
};
__device__ __forceinline__ ChunkAt chunk_at(const ScanP& p, uint32_t slot) {
    ChunkAt c;
    if (!p.cu) {
        uint32_t u = slot;
        c.ch = take(u, (p.T + kQ - 1) / kQ);
        c.b = static_cast<int>(u);
    } else {  // the last b with b + begin_b / 64 <= slot, eight boundaries a step
        int lo = 0, n = p.B;
        while (n > 1) {
            const int step = (n + 7) / 8;
            uint32_t at[7];
            int k = 0;
#pragma unroll
            for (int i = 0; i < 7; i++) {
                const int b = lo + (step * (i + 1) < n ? step * (i + 1) : 0);
                at[i] = static_cast<uint32_t>(b + packed_span(p.cu, b, p.T).begin / kQ);
            }
#pragma unroll
            for (int i = 0; i < 7; i++) k = step * (i + 1) < n && at[i] <= slot ? i + 1 : k;
            lo += k * step;
            n = n - k * step < step ? n - k * step : step;
        }
        c.b = lo;
        c.ch = static_cast<int>(slot) - lo - packed_span(p.cu, lo, p.T).begin / kQ;
    }
    c.sr = c.b < p.B ? seq_range(p, c.b) : SeqRange{0, 0};
    c.used = c.ch >= 0 && c.ch < (c.sr.len + kQ - 1) / kQ;
    return c;
}

// Every chunk's decays, a wave each; read by the walks, the gradients and the rates' gradients.
__global__ __launch_bounds__(256) void decays_kernel(ScanP p, Decay* out, uint32_t slots) {
    __shared__ __align__(16) Decay d[4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t slot = blockIdx.x * 4u + wave;
    const int h = take(slot, p.H);
    if (slot >= slots) return;
    const ChunkAt at = chunk_at(p, slot);
    if (!at.used) return;
    const int live = at.sr.len - at.ch * kQ;
    DtAhead dt;
    dt.fetch(p, at.sr.begin + static_cast<int64_t>(at.ch) * kQ, h, lane, live);
    make_decay(d[wave], dt.value(p) + (p.bias ? p.bias[h] : 0.0f), p.softplus, live, p.A[h]);
    uv4* o = reinterpret_cast<uv4*>(out + static_cast<int64_t>(slot) * p.H + h);
#pragma unroll
    for (int q = 0; q < 2; q++) o[lane + 64 * q] = reinterpret_cast<const uv4*>(&d[wave])[lane + 64 * q];
}

template <class T, int N>
struct WalkLds {
    T b[kQ * lds_row<T>(N)];
    T x[kQ * lds_row64<T>()];
    Decay d;
};

// Both directions of the state's walk for 64 value columns of a head, a workgroup each in one
// launch (they are independent, and the chip holds two a CU).  Forward: S from b, x and W, the
// state entering each chunk to `S`.  Back: dS from c, dy and exp(cum), the gradient of the state
// leaving each chunk to `dS`, and dS0.  ONE: a workgroup a chunk, its own contribution from zero
// only (joined by walk_join_kernel): for few heads.
// The state is held transposed (a lane: one row, four consecutive columns of each tile), so
// that it is stored in 16-byte pieces.
template <class T, int N, bool ONE>
__global__ __launch_bounds__(256) void scan_walk_kernel(ScanP p, const T* dy, const float* S0, const float* dST, float* Sst,
                                                        float* dSst, const Decay* decays, float* dS0) {
    using MT = Mat<T>;
    constexpr int P3 = MT::template parts<3>;
    constexpr int RB = lds_row<T>(N), RX = lds_row64<T>();
    __shared__ __align__(16) WalkLds<T, N> lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lm = lane & 15, g = lane >> 4;

    const int tiles = p.dv / kPT;
    uint32_t u = die_unit(blockIdx.x, gridDim.x);
    const bool rev = take(u, 2) != 0;
    const int tile = take(u, tiles), h = take(u, p.H);
    const float* first = rev ? dST : S0;
    float* states = rev ? dSst : Sst;
    float* last = rev ? dS0 : nullptr;
    const int64_t ld_x = rev ? static_cast<int64_t>(p.H) * p.dv : p.ld_x;
    int bi = static_cast<int>(u), only = 0;  // (ONE: u is a slot)
    SeqRange sr;
    if constexpr (ONE) {
        const ChunkAt at = chunk_at(p, u);
        if (!at.used) return;
        bi = at.b, only = at.ch, sr = at.sr;
    } else {
        sr = seq_range(p, bi);
    }
    const int nch = (sr.len + kQ - 1) / kQ;
    const int steps = ONE ? 1 : nch;
    const int grp = h / (p.H / p.G);
    const int col = tile * kPT + 16 * wave + 4 * g;  // this lane's four columns
    const size_t head = static_cast<size_t>(p.dk) * p.dv;

    f4 S[N / 16];
#pragma unroll
    for (int i = 0; i < N / 16; i++) {
        const int n = 16 * i + lm;
        S[i] = f4{};
        if (!ONE && first && n < p.dk)
            S[i] = *reinterpret_cast<const f4*>(first + (static_cast<size_t>(bi) * p.H + h) * head + static_cast<size_t>(n) * p.dv + col);
    }
    auto put = [&](float* at) {
#pragma unroll
        for (int i = 0; i < N / 16; i++) {
            const int n = 16 * i + lm;
            if (n < p.dk) *reinterpret_cast<f4*>(at + static_cast<size_t>(n) * p.dv + col) = S[i];
        }
    };
    const T* xg = (rev ? dy : static_cast<const T*>(p.x)) + static_cast<int64_t>(h) * p.dv + tile * kPT;
    const T* bg = static_cast<const T*>(rev ? p.c : p.b) + static_cast<int64_t>(grp) * p.dk;
    const int64_t ld_b = rev ? p.ld_c : p.ld_b;
    Tile<T, N, 256> tb;
    Tile<T, kPT, 256> tx;
    DecayAhead<256> td;
    auto at_step = [&](int i) { return ONE ? only : rev ? nch - 1 - i : i; };
    auto fetch = [&](int ch) {
        const int64_t row0 = sr.begin + static_cast<int64_t>(ch) * kQ;
        const int live = sr.len - ch * kQ;
        tb.load(bg + row0 * ld_b, ld_b, live, p.dk);
        tx.load(xg + row0 * ld_x, ld_x, live, kPT);
        td.load(decays + slot_of(p, bi, sr.begin, ch) * p.H + h);
    };
    if (steps > 0) fetch(at_step(0));
    for (int i = 0; i < steps; i++) {
        const int ch = at_step(i);
        tb.store(lds.b, RB);
        tx.store(lds.x, RX);
        td.store(lds.d);
        __syncthreads();
        if (i + 1 < steps) fetch(at_step(i + 1));
        float* slot = states + (static_cast<size_t>(slot_of(p, bi, sr.begin, ch)) * p.H + h) * head;
        if (!ONE) put(slot);
        typename MT::Frag wx[2][P3];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            float v[8];
            MT::widen8(MT::col8(lds.x, RX, 32 * k, 16 * wave, lane), v);
            float wt[8];
            get8((rev ? lds.d.head : lds.d.w) + 32 * k + 8 * g, wt);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] *= wt[j];
            MT::template split<P3>(v, wx[k]);
        }
        const float total = lds.d.total[0];
#pragma unroll
        for (int n = 0; n < N / 16; n++) S[n] *= total;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            typename MT::Frag bf[N / 16];
#pragma unroll
            for (int n = 0; n < N / 16; n++) bf[n] = MT::col8(lds.b, RB, 32 * k, 16 * n, lane);
#pragma unroll
            for (int q = 0; q < P3; q++)
#pragma unroll
                for (int n = 0; n < N / 16; n++) S[n] = MT::mma(wx[k][q], bf[n], S[n]);
        }
        if (ONE) put(slot);
        __syncthreads();
    }
    if (!ONE && last) put(last + (static_cast<size_t>(bi) * p.H + h) * head);
}

// From the chunks' own contributions, in place: the state that enters each of them and (y = 1)
// the gradient of the state that leaves it.
__global__ __launch_bounds__(256) void walk_join_kernel(ScanP p, const float* S0, const float* dST, float* Sst, float* dSst,
                                                        const Decay* decays, float* dS0) {
    const bool rev = blockIdx.y != 0;
    const float* first = rev ? dST : S0;
    float* states = rev ? dSst : Sst;
    float* last = rev ? dS0 : nullptr;
    const int per = p.dk * p.dv / 4;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<int64_t>(p.B) * p.H * per) return;
    const int e = static_cast<int>(i % per);
    const int64_t bh = i / per;
    const int h = static_cast<int>(bh % p.H), bi = static_cast<int>(bh / p.H);
    const SeqRange sr = seq_range(p, bi);
    const int nch = (sr.len + kQ - 1) / kQ;
    fv4 S = {};
    if (first) S = reinterpret_cast<const fv4*>(first)[bh * per + e];
    for (int k0 = 0; k0 < nch; k0 += 8) {  // eight chunks' loads in flight: only the sums are a chain
        fv4 own[8];
        float total[8];
        fv4* l[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int k = k0 + j < nch ? k0 + j : nch - 1;
            const int64_t at = slot_of(p, bi, sr.begin, rev ? nch - 1 - k : k) * p.H + h;
            l[j] = reinterpret_cast<fv4*>(states) + at * per + e;
            own[j] = *l[j];
            total[j] = decays[at].total[0];
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (k0 + j >= nch) break;
            *l[j] = S;
            S = S * total[j] + own[j];
        }
    }
    if (last) reinterpret_cast<fv4*>(last)[bh * per + e] = S;
}

// What the decays' gradients of one chunk and head are formed from: FP32 sums over a wave's part of
// a row or column, joined in double for 0.6% of the time.  Against their 64-bit values, beside the same
// formulas in FP32 tensor operations with sums over tokens in double: dA and ddt_bias of 8 x 4096
// bf16 tokens and 16 heads 0.6 times as far (joined in FP32 up to 2.5 times); FP32 inputs, the means
// over six seeds 0.3 to 0.8 times, ddt_bias of two heads 1.8 times, single seeds 0.1 to 8 times (few
// sums, which nearly cancel).  dD 1.5 to 5 times: a token's 64 columns are added in FP32.
struct RateSums {
    double r[kQ], c[kQ], inner[kQ];  // r_t, c_t, and c_t's part from dS
    double sd, dd;                   // <S, dS>, sum of dy x
    float diag[kQ];                  // P's diagonal
};

template <class T, int N>
struct GradLds {
    T b[kQ * lds_row<T>(N)];
    T c[kQ * lds_row<T>(N)];
    T x[kQ * lds_row64<T>()];
    T dy[kQ * lds_row64<T>()];
    // M[t][s] and dG[t][s], as two bf16 parts: 2^-17 of a value for bf16 results (rounded to one,
    // db and dc were 1.4 times as far from their 64-bit values as their own rounding leaves them)
    T m[Mat<T>::template parts<2>][kQ * lds_row64<T>()];
    T dg[Mat<T>::template parts<2>][kQ * lds_row64<T>()];
    T ds[sizeof(T) == 2 ? 2 : 1][sizeof(T) == 2 ? N * lds_row64<T>() : 8];  // dS (two bf16 parts); FP32 reads it from memory
    Decay d;
    // partial sums of the decays' gradients, by parity of the iteration (they are joined beside the next)
    float rt[2][10][16], ct[2][10][16];          // the pair tiles' row and column sums
    float ri[2][N / 16][kQ], ci[2][N / 16][kQ];  // sums over 16 state rows
    float sd[2][8];                              // the waves' <S, dS>
    float pd[2][kQ], dd[2][kQ];                  // the diagonals of P and dM
};

__device__ __forceinline__ void lower_tile_of(int k, int& ti, int& si) {
    ti = k < 1 ? 0 : k < 3 ? 1 : k < 6 ? 2 : 3;
    si = k - ti * (ti + 1) / 2;
}

// Gradients of one chunk for one slice of a group's heads, by eight waves; a head's 64 value
// columns an iteration.  Pairs: the ten lower tiles over the waves, and beside them the last
// iteration's sums for the decays' gradients.  dX: a wave 16 columns by 32 tokens.  dC, dB: a
// wave 16 state rows by all tokens (fewer rows than 128: by a part of them), kept in registers
// over the heads.  Memory, LDS (conflicts in 19% of the cycles) and the vector units (41%) share
// the time: b^T and c^T, which do not change over the heads, stay in registers, and the next
// iteration's loads are issued in three places.  dbp, dcp: FP32 partial sums of db and dc per
// slice ([slice][row][G][dk]), or null where one slice holds the whole group.
template <class T, int N>
__global__ __launch_bounds__(512) void scan_grad_kernel(ScanP p, const T* dyr, const float* Sin, const float* dSe, void* dx_,
                                                        void* db_, void* dc_, float* dbp, float* dcp, const Decay* decays,
                                                        RateSums* sums, int slices, int64_t rows) {
    using MT = Mat<T>;
    // S and dS as operands: three bf16 parts (exact) where the decays' gradients come from them,
    // two of dS for dX
    constexpr int P2 = MT::template parts<2>, P3 = MT::template parts<3>;
    constexpr int RB = lds_row<T>(N), RX = lds_row64<T>(), RM = lds_row64<T>();
    constexpr int KS = N / 32, NTL = N / 16, PARTS = 8 / NTL, TI = 4 / PARTS;
    extern __shared__ __align__(16) char raw_lds[];
    GradLds<T, N>& lds = *reinterpret_cast<GradLds<T, N>*>(raw_lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lm = lane & 15, g = lane >> 4;
    const int nt = PARTS == 1 ? wave : wave % NTL, n0 = 16 * nt, part = PARTS == 1 ? 0 : wave / NTL;  // state rows and token part of dC, dB
    constexpr int kJoin = 7;                              // the wave that joins the sums

    uint32_t u = die_unit(blockIdx.x, gridDim.x);
    const int slice = take(u, slices), grp = take(u, p.G);
    const uint32_t slot = u;
    const ChunkAt at = chunk_at(p, slot);
    if (!at.used) return;
    const SeqRange sr = at.sr;
    const int64_t row0 = sr.begin + static_cast<int64_t>(at.ch) * kQ;
    const int live = sr.len - at.ch * kQ < kQ ? sr.len - at.ch * kQ : kQ;

    const int hpg = __builtin_amdgcn_readfirstlane(p.H / p.G), per = __builtin_amdgcn_readfirstlane((hpg + slices - 1) / slices);
    const int h0 = grp * hpg + slice * per;
    const int h1 = slice * per + per < hpg ? h0 + per : (grp + 1) * hpg;
    const int tiles = p.dv / kPT;
    const size_t head = static_cast<size_t>(p.dk) * p.dv;
    const int iters = (h1 - h0) * tiles;

    Tile<T, kPT, 512> tx, ty;
    DecayAhead<512> td;
    float Sr[2][8], dSr[2][8];
    auto fetch_rows = [&](int it) {
        uint32_t q = static_cast<uint32_t>(it);
        const int tile = take(q, tiles), h = h0 + static_cast<int>(q);
        tx.load(static_cast<const T*>(p.x) + row0 * p.ld_x + static_cast<int64_t>(h) * p.dv + tile * kPT, p.ld_x, live, kPT);
        ty.load(dyr + (row0 * p.H + h) * p.dv + tile * kPT, static_cast<int64_t>(p.H) * p.dv, live, kPT);
        td.load(decays + static_cast<int64_t>(slot) * p.H + h);
    };
    const int soff = n0 + lm < p.dk ? ((n0 + lm) * p.dv + 8 * g) * 4 : -1024;
    auto fetch_state = [&](int it, const float* from, float (&to)[2][8]) {
        uint32_t q = static_cast<uint32_t>(it);
        const int tile = take(q, tiles);
        const size_t at = (static_cast<size_t>(slot) * p.H + h0 + q) * head + tile * kPT;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(from + at, head * 4);
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const f4 v = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, soff, 128 * k + 16 * i, 0));
#pragma unroll
                for (int j = 0; j < 4; j++) to[k][4 * i + j] = v[j];
            }
    };
    fetch_rows(0);
    fetch_state(0, Sin, Sr);
    fetch_state(0, dSe, dSr);
    {  // this chunk's b and c, and zeros above the diagonals
        Tile<T, N, 512> t;
        t.load(static_cast<const T*>(p.b) + row0 * p.ld_b + static_cast<int64_t>(grp) * p.dk, p.ld_b, live, p.dk);
        t.store(lds.b, RB);
        t.load(static_cast<const T*>(p.c) + row0 * p.ld_c + static_cast<int64_t>(grp) * p.dk, p.ld_c, live, p.dk);
        t.store(lds.c, RB);
        for (int i = threadIdx.x; i < P2 * kQ * RM; i += 512) {
            (&lds.m[0][0])[i] = T{};
            (&lds.dg[0][0])[i] = T{};
        }
    }
    __syncthreads();
    f4 G[2];  // G^T of this wave's lower tiles: rows s, columns t
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const int k = wave + 8 * q;
        G[q] = f4{};
        if (k < 10) {
            int ti, si;
            lower_tile_of(k, ti, si);
#pragma unroll
            for (int ks = 0; ks < KS; ks++)
                G[q] = MT::mma(MT::row8(lds.b + (16 * si + lm) * RB + 32 * ks + 8 * g),
                               MT::row8(lds.c + (16 * ti + lm) * RB + 32 * ks + 8 * g), G[q]);
        }
    }
    typename MT::Frag bT[2], cT[2];  // b^T, c^T: row n0 + lm, tokens 32 k + 8 g ..
#pragma unroll
    for (int k = 0; k < 2; k++) {
        bT[k] = MT::col8(lds.b, RB, 32 * k, n0, lane);
        cT[k] = MT::col8(lds.c, RB, 32 * k, n0, lane);
    }
    f4 dC[TI] = {}, dB[TI] = {};  // rows n, columns t (s)

    // kJoin: iteration it's partial sums, added up over a head's tiles; lane = token
    double racc = 0.0, cacc = 0.0, iacc = 0.0, sdacc = 0.0, ddacc = 0.0;
    float pdacc = 0.0f;
    auto join = [&](int it) {
        const int par = it & 1;
        const int tq = lane >> 4, tl = lane & 15;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const float rt = lds.rt[par][tq * (tq + 1) / 2 + (q <= tq ? q : 0)][tl], ct = lds.ct[par][(q >= tq ? q * (q + 1) / 2 : 0) + tq][tl];
            racc += q <= tq ? rt : 0.0f;
            cacc += q >= tq ? ct : 0.0f;
        }
        double inner = 0.0;
#pragma unroll 2
        for (int q = 0; q < NTL; q++) {  // (unrolled whole, its registers would spill others)
            racc += lds.ri[par][q][lane];
            inner += lds.ci[par][q][lane];
        }
        cacc += inner;
        iacc += inner;
        pdacc += lds.pd[par][lane];
        ddacc += lds.dd[par][lane];
        sdacc += lds.sd[par][lane & 7];  // lane q: wave q's
        uint32_t q = static_cast<uint32_t>(it);
        if (take(q, tiles) != tiles - 1) return;
        RateSums& o = sums[slot * p.H + h0 + q];
        o.r[lane] = racc;
        o.c[lane] = cacc;
        o.inner[lane] = iacc;
        o.diag[lane] = pdacc;
        const double sd = wave_last(wave_prefix(lane < 8 ? sdacc : 0.0)), dd = wave_last(wave_prefix(ddacc));
        if (lane == 0) {
            o.sd = sd;
            o.dd = dd;
        }
        racc = cacc = iacc = sdacc = ddacc = 0.0;
        pdacc = 0.0f;
    };

    for (int it = 0; it < iters; it++) {
        uint32_t qh = static_cast<uint32_t>(it);
        const int tile = take(qh, tiles), h = h0 + static_cast<int>(qh), par = it & 1;
        const Decay& d = lds.d;
        const float Dh = p.D ? p.D[h] : 0.0f;
        const int next = it + 1 < iters ? it + 1 : it;
        // (The lane's indices are made opaque in every part: addresses formed from them before the
        // loop would fill the registers.)
        // ---- this head's tiles to LDS, S and dS as operands (row n0 + lm, columns 32 k + 8 g ..)
        tx.store(lds.x, RX);
        ty.store(lds.dy, RX);
        td.store(lds.d);
        typename MT::Frag Sf[2][P3], dSf[2][P3];
        float sd = 0.0f;
        {
        const int ln = opaque(lane), lm = ln & 15, g = ln >> 4;
#pragma unroll
        for (int k = 0; k < 2; k++) {
#pragma unroll
            for (int j = 0; j < 8; j++) sd = __builtin_fmaf(Sr[k][j], dSr[k][j], sd);
            MT::template split<P3>(Sr[k], Sf[k]);
            MT::template split<P3>(dSr[k], dSf[k]);
            if constexpr (sizeof(T) == 2) {
                if (part == 0) {
#pragma unroll
                    for (int r = 0; r < P2; r++)
                        *reinterpret_cast<typename MT::Frag*>(&lds.ds[r][(n0 + lm) * RX + 32 * k + 8 * g]) = dSf[k][r];
                }
            }
        }
        sd = part == 0 ? wave_sum(sd) : 0.0f;
        if (lane == 0) lds.sd[par][wave] = sd;
        }
        __syncthreads();

        // ---- pairs: dM^T tiles (rows s, columns t)
        if (sizeof(T) == 2) fetch_state(next, Sin, Sr);  // (FP32: no registers to hold it so early)
        {
        const int ln = opaque(lane), lm = ln & 15, g = ln >> 4;
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const int k = wave + 8 * q;
            if (k >= 10) continue;
            int ti, si;
            lower_tile_of(k, ti, si);
            const int t = 16 * ti + lm, s0 = 16 * si + 4 * g;
            typename MT::Frag xf[2], yf[2];
#pragma unroll
            for (int ks = 0; ks < 2; ks++) {
                xf[ks] = MT::row8(lds.x + (16 * si + lm) * RX + 32 * ks + 8 * g);
                yf[ks] = MT::row8(lds.dy + t * RX + 32 * ks + 8 * g);
            }
            const float thi = d.hi[t], tlo = d.lo[t];
            const f4 shi = *reinterpret_cast<const f4*>(d.hi + s0), slo = *reinterpret_cast<const f4*>(d.lo + s0);
            const f4 sdl = *reinterpret_cast<const f4*>(d.delta + s0);
            f4 acc = {};
#pragma unroll
            for (int ks = 0; ks < 2; ks++) acc = MT::mma(xf[ks], yf[ks], acc);
            float m[4], dg[4], pc[4], pr = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int s = s0 + r;
                const float L = s <= t ? pair_decay(thi, tlo, shi[r], slo[r]) : 0.0f;
                const float gl = G[q][r] * L, dl = sdl[r];
                m[r] = gl * dl;
                dg[r] = L * dl * acc[r];
                pc[r] = s < t ? gl * acc[r] : 0.0f;
                pr = __builtin_fmaf(pc[r], dl, pr);
                if (s == t) {
                    lds.dd[par][t] = acc[r];
                    lds.pd[par][t] = gl * acc[r];
                }
            }
            MT::template put4<P2>(&lds.m[0][t * RM + s0], kQ * RM, m);
            MT::template put4<P2>(&lds.dg[0][t * RM + s0], kQ * RM, dg);
            pr = rows_sum(pr);
            if (g == 0) lds.rt[par][k][lm] = pr;
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const float s = group_sum<16>(pc[r]);
                if (lm == 0) lds.ct[par][k][4 * g + r] = s;
            }
        }
        }
        if (wave == kJoin && it > 0) join(it - 1);
        __syncthreads();

        // ---- dX^T: rows: columns pc + 4 g + r; column: s
        if (sizeof(T) == 2) fetch_state(next, dSe, dSr);
        {
            const int ln = opaque(lane), lm = ln & 15, g = ln >> 4;
            const int pc = 16 * (wave & 3), half = wave >> 2;
            f4 acc[2] = {};
#pragma unroll
            for (int k1 = 0; k1 < KS; k1 += 2) {
                typename MT::Frag dsT[2][P2], bf[2][2];
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    const int ks = k1 + q;
                    if (ks >= KS) continue;
#pragma unroll
                    for (int j = 0; j < 2; j++) bf[q][j] = MT::row8(lds.b + (32 * half + 16 * j + lm) * RB + 32 * ks + 8 * g);
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int k = 0; k < P2; k++) dsT[q][k] = MT::col8(lds.ds[k], RX, 32 * ks, pc, ln);
                    } else {
                        const float* src = dSe + (static_cast<size_t>(slot) * p.H + h) * head + tile * kPT + pc + lm;
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const int n = 32 * ks + 8 * g + j;
                            dsT[q][0][j] = n < p.dk ? src[static_cast<size_t>(n) * p.dv] : 0.0f;
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int q = 0; q < 2; q++)
#pragma unroll
                    for (int k = 0; k < P2; k++)
#pragma unroll
                        for (int j = 0; j < 2; j++)
                            if (k1 + q < KS) acc[j] = MT::mma(dsT[q][k], bf[q][j], acc[j]);
            }
            typename MT::Frag dyT[2], mf[2][P2][2];
#pragma unroll
            for (int ks = 0; ks < 2; ks++) {
                dyT[ks] = MT::col8(lds.dy, RX, 32 * ks, pc, ln);
#pragma unroll
                for (int k = 0; k < P2; k++)
#pragma unroll
                    for (int j = 0; j < 2; j++) mf[ks][k][j] = MT::col8(lds.m[k], RM, 32 * ks, 32 * half + 16 * j, ln);
            }
            // (rows behind the sequence lie behind the buffer's end)
            const __amdgpu_buffer_rsrc_t rdx =
                make_rsrc(static_cast<T*>(dx_) + row0 * p.ld_x + static_cast<int64_t>(h) * p.dv + tile * kPT, live * p.ld_x * sizeof(T));
            float w[2];
#pragma unroll
            for (int j = 0; j < 2; j++) w[j] = d.w[32 * half + 16 * j + lm];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 2; j++) acc[j] *= w[j];
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
#pragma unroll
                for (int k = 0; k < P2; k++)
#pragma unroll
                    for (int j = 0; j < 2; j++)
                        if (ks >= half) acc[j] = MT::mma(dyT[ks], mf[ks][k][j], acc[j]);  // (tokens before s: zero)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int s = 32 * half + 16 * j + lm;
                float yv[4];
                MT::get4(lds.dy + s * RX + pc + 4 * g, yv);
#pragma unroll
                for (int r = 0; r < 4; r++) acc[j][r] = __builtin_fmaf(Dh, yv[r], acc[j][r]);
                const int off = (s * static_cast<int>(p.ld_x) + pc + 4 * g) * static_cast<int>(sizeof(T));
                if constexpr (sizeof(T) == 2)
                    __builtin_amdgcn_raw_buffer_store_b64(uv2{pack16(acc[j][0], acc[j][1]), pack16(acc[j][2], acc[j][3])}, rdx, off, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uv4, acc[j]), rdx, off, 0, 0);
            }
        }
        // ---- dC^T, dB^T: rows n of this wave, columns t, s
        fetch_rows(next);
        {
            const int ln = opaque(lane), lm = ln & 15, g = ln >> 4;
            float ri[TI], ci[TI];
#pragma unroll
            for (int ii = 0; ii < TI; ii++) {
                const int i = part * TI + ii, t = 16 * i + lm;
                __builtin_amdgcn_sched_barrier(0);
                typename MT::Frag yf[2], xf[2], gr[2][P2], gc[2][P2];
#pragma unroll
                for (int ks = 0; ks < 2; ks++) {
                    yf[ks] = MT::row8(lds.dy + t * RX + 32 * ks + 8 * g);
                    xf[ks] = MT::row8(lds.x + t * RX + 32 * ks + 8 * g);
#pragma unroll
                    for (int k = 0; k < P2; k++) {
                        gr[ks][k] = MT::row8(&lds.dg[k][t * RM + 32 * ks + 8 * g]);
                        gc[ks][k] = MT::col8(lds.dg[k], RM, 32 * ks, 16 * i, ln);
                    }
                }
                float cv[4], bv[4];
                MT::get4(lds.c + t * RB + n0 + 4 * g, cv);
                MT::get4(lds.b + t * RB + n0 + 4 * g, bv);
                const float head_t = d.head[t], tail_t = d.tail[t], w_t = d.w[t];
                __builtin_amdgcn_sched_barrier(0);
                f4 a = {}, b = {};
#pragma unroll
                for (int ks = 0; ks < 2; ks++)
#pragma unroll
                    for (int k = 0; k < P3; k++) {
                        a = MT::mma(Sf[ks][k], yf[ks], a);
                        b = MT::mma(dSf[ks][k], xf[ks], b);
                    }
#pragma unroll
                for (int ks = 0; ks < 2; ks++)
#pragma unroll
                    for (int k = 0; k < P2; k++) {
                        if (ks <= i / 2) dC[ii] = MT::mma(bT[ks], gr[ks][k], dC[ii]);
                        if (ks >= i / 2) dB[ii] = MT::mma(cT[ks], gc[ks][k], dB[ii]);
                    }
                ri[ii] = ci[ii] = 0.0f;
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    ri[ii] = __builtin_fmaf(a[r], cv[r], ri[ii]);
                    ci[ii] = __builtin_fmaf(b[r], bv[r], ci[ii]);
                    dC[ii][r] = __builtin_fmaf(a[r], head_t, dC[ii][r]);
                    dB[ii][r] = __builtin_fmaf(b[r], w_t, dB[ii][r]);
                }
                ri[ii] *= head_t;
                ci[ii] *= tail_t;
            }
            if constexpr (TI == 4) {  // lane group g is left with the sums of tile g
                const float r = rows_scatter4(ri), c = rows_scatter4(ci);
                lds.ri[par][nt][16 * g + lm] = r;
                lds.ci[par][nt][16 * g + lm] = c;
            } else {
#pragma unroll
                for (int ii = 0; ii < TI; ii++) {
                    const float r = rows_sum(ri[ii]), c = rows_sum(ci[ii]);
                    if (g == 0) {
                        lds.ri[par][nt][16 * (part * TI + ii) + lm] = r;
                        lds.ci[par][nt][16 * (part * TI + ii) + lm] = c;
                    }
                }
            }
        }
        if (sizeof(T) == 4) {
            fetch_state(next, Sin, Sr);
            fetch_state(next, dSe, dSr);
        }
        __syncthreads();
    }
    if (wave == kJoin) join(iters - 1);
    // ---- db, dc
    const int n = n0 + 4 * g;
    if (n >= p.dk) return;
#pragma unroll
    for (int ii = 0; ii < TI; ii++) {
        const int t = 16 * (part * TI + ii) + lm;
        if (t >= live) continue;
        const float vb[4] = {dB[ii][0], dB[ii][1], dB[ii][2], dB[ii][3]};
        const float vc[4] = {dC[ii][0], dC[ii][1], dC[ii][2], dC[ii][3]};
        if (dbp) {
            const size_t at = ((static_cast<size_t>(slice) * rows + row0 + t) * p.G + grp) * p.dk + n;
            *reinterpret_cast<f4*>(dbp + at) = dB[ii];
            *reinterpret_cast<f4*>(dcp + at) = dC[ii];
        } else {
            MT::template put4<1>(static_cast<T*>(db_) + (row0 + t) * p.ld_b + static_cast<int64_t>(grp) * p.dk + n, 0, vb);
            MT::template put4<1>(static_cast<T*>(dc_) + (row0 + t) * p.ld_c + static_cast<int64_t>(grp) * p.dk + n, 0, vc);
        }
    }
}

// db and dc from the slices' partial sums, in slice order.
template <class T>
__global__ __launch_bounds__(256) void join_slices_kernel(ScanP p, const float* dbp, const float* dcp, T* db, T* dc,
                                                          int slices, int64_t rows) {
    const int per = p.G * p.dk / 4;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= rows * per) return;
    const int64_t row = i / per;
    const int e = static_cast<int>(i % per) * 4;
    if (p.cu) {  // rows outside every sequence are cleared by their own kernel
        const int b = packed_find(p.cu, p.B, static_cast<int>(row));
        const Span s = packed_span(p.cu, b, p.T);
        if (row < s.begin || row >= s.end) return;
    }
    fv4 vb = {}, vc = {};
    for (int s = 0; s < slices; s++) {
        vb += *reinterpret_cast<const fv4*>(dbp + (s * rows + row) * per * 4 + e);
        vc += *reinterpret_cast<const fv4*>(dcp + (s * rows + row) * per * 4 + e);
    }
    const float fb[4] = {vb[0], vb[1], vb[2], vb[3]}, fc[4] = {vc[0], vc[1], vc[2], vc[3]};
    Mat<T>::template put4<1>(db + row * p.ld_b + e, 0, fb);
    Mat<T>::template put4<1>(dc + row * p.ld_c + e, 0, fc);
}

// Zero gradients for a packing's tokens outside every sequence, 256 tokens a workgroup.
template <class T>
__global__ __launch_bounds__(256) void clear_outside_kernel(ScanP p, T* dx, void* ddt, T* db, T* dc) {
    __shared__ bool outside[256];
    const int t0 = static_cast<int>(blockIdx.x) * 256, tid = threadIdx.x;
    const int n = p.T - t0 < 256 ? p.T - t0 : 256;
    bool out = false;
    if (tid < n) {
        const Span s = packed_span(p.cu, packed_find(p.cu, p.B, t0 + tid), p.T);
        out = t0 + tid < s.begin || t0 + tid >= s.end;
    }
    outside[tid] = out;
    if (__syncthreads_count(out) == 0) return;
    for (int k = 0; k < n; k++) {
        if (!outside[k]) continue;
        const int64_t t = t0 + k;
        for (int i = tid; i < p.H * p.dv; i += 256) dx[t * p.ld_x + i] = T{};
        for (int i = tid; i < p.G * p.dk; i += 256) {
            db[t * p.ld_b + i] = T{};
            dc[t * p.ld_c + i] = T{};
        }
        for (int i = tid; i < p.H; i += 256) store_elem(ddt, t * p.ld_dt + i, p.dt_dtype, 0.0f);
    }
}

// The decays' gradients of every chunk, a wave each: the suffix sums of r_t - Delta_t c_t and what
// the last token gets from the chunk's end, in double (the terms cancel); ddt, and the chunk's
// share of dA, dD and ddt_bias to hp [slot][3][H].
__global__ __launch_bounds__(256) void rates_kernel(ScanP p, const Decay* decays, const RateSums* sums, void* ddt, double* hp, uint32_t slots) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t su = blockIdx.x * 4u + wave;
    const int h = take(su, p.H);
    if (su >= slots) return;
    const int64_t slot = su;
    double* o = hp + slot * 3 * p.H + h;
    const ChunkAt at = chunk_at(p, su);
    if (!at.used) {
        if (lane < 3) o[lane * p.H] = 0.0;
        return;
    }
    const SeqRange sr = at.sr;
    const int ch = at.ch, live = sr.len - ch * kQ;
    const Decay& d = decays[slot * p.H + h];
    const RateSums& m = sums[slot * p.H + h];
    const double delta = d.delta[lane], c = m.c[lane];
    double v = m.r[lane] - delta * c;
    const double into = wave_last(wave_prefix(delta * m.inner[lane]));
    if (lane == 63) v += static_cast<double>(d.total[0]) * m.sd + into;
    const double pre = wave_prefix(v);
    const double rate = wave_last(pre) - pre + v;  // the log decay's gradient
    const float dd = static_cast<float>(c + static_cast<double>(m.diag[lane]) + static_cast<double>(p.A[h]) * rate);
    const float dz = lane < live ? (p.softplus ? dd * sigmoid_full(d.z[lane]) : dd) : 0.0f;
    if (lane < live) store_elem(ddt, (sr.begin + static_cast<int64_t>(ch) * kQ + lane) * p.ld_dt + h, p.dt_dtype, dz);
    const double da = wave_last(wave_prefix(rate * delta)), db = wave_last(wave_prefix(static_cast<double>(dz)));
    if (lane == 0) {
        o[0] = da;
        o[p.H] = m.dd;
        o[2 * p.H] = db;
    }
}

// The heads' dA, dD and ddt_bias over all chunks (a packing's unused slots hold zeros).
__global__ __launch_bounds__(256) void head_sums_kernel(ScanP p, const double* hp, int64_t slots, float* dA, float* dD, float* dbias) {
    __shared__ double red[256];
    const int h = blockIdx.x % p.H, which = blockIdx.x / p.H;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < slots; i += 256) s += hp[i * 3 * p.H + static_cast<int64_t>(which) * p.H + h];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int n = 128; n > 0; n >>= 1) {
        if (threadIdx.x < n) red[threadIdx.x] += red[threadIdx.x + n];
        __syncthreads();
    }
    float* out = which == 0 ? dA : which == 1 ? dD : dbias;
    if (threadIdx.x == 0 && out) out[h] = static_cast<float>(red[0]);
}

__global__ __launch_bounds__(256) void copy_or_zero_kernel(const float* src, float* dst, int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
        dst[i] = src ? src[i] : 0.0f;
}

// Slices of a group's heads: enough workgroups for two a CU.
int grad_slices(const la_scan_config& c, bool packed) {
    const int64_t units = slot_count(c, packed) * c.G;
    const int hpg = c.H / c.G;
    if (units == 0 || hpg == 0) return 1;
    int64_t n = (512 + units - 1) / units;
    if (n > hpg) n = hpg;
    const int per = static_cast<int>((hpg + n - 1) / n);
    return (hpg + per - 1) / per;
}

struct BwdWs {
    size_t S, dS, decays, sums, dbp, dcp, hp, total;
};
BwdWs bwd_ws(const la_scan_config& c, bool packed) {
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const int64_t slots = slot_count(c, packed), rows = packed ? c.T : static_cast<int64_t>(c.B) * c.T;
    const size_t st = up(static_cast<size_t>(slots) * c.H * c.d_k * c.d_v * sizeof(float));
    const int slices = grad_slices(c, packed);
    const size_t bc = slices > 1 ? up(static_cast<size_t>(slices) * rows * c.G * c.d_k * sizeof(float)) : 0;
    BwdWs w;
    w.S = 0;
    w.dS = w.S + st;
    w.decays = w.dS + st;
    w.sums = w.decays + up(static_cast<size_t>(slots) * c.H * sizeof(Decay));
    w.dbp = w.sums + up(static_cast<size_t>(slots) * c.H * sizeof(RateSums));
    w.dcp = w.dbp + bc;
    w.hp = w.dcp + bc;
    w.total = w.hp + up(static_cast<size_t>(slots) * 3 * c.H * sizeof(double));
    return w;
}

template <class T, int N>
hipError_t launch(const la_scan_config& c, const ScanArgs& a, hipStream_t s) {
    const ScanP p = scan_params(c, a);
    const bool packed = a.cu != nullptr;
    const BwdWs w = bwd_ws(c, packed);
    float* S = reinterpret_cast<float*>(a.ws + w.S);
    float* dS = reinterpret_cast<float*>(a.ws + w.dS);
    Decay* decays = reinterpret_cast<Decay*>(a.ws + w.decays);
    RateSums* sums = reinterpret_cast<RateSums*>(a.ws + w.sums);
    double* hp = reinterpret_cast<double*>(a.ws + w.hp);
    const int64_t rows = a.cu ? c.T : static_cast<int64_t>(c.B) * c.T;
    const int64_t slots = slot_count(c, packed), tiles = c.d_v / kPT;
    const int64_t groups = static_cast<int64_t>(c.B) * c.H * tiles, chunks = slots * c.H * tiles;
    const T* dy = static_cast<const T*>(a.dy);
    const unsigned units = static_cast<unsigned>((slots * c.H + 3) / 4);
    decays_kernel<<<dim3(units), 256, 0, s>>>(p, decays, static_cast<uint32_t>(slots));
    // Enough heads: a workgroup walks a sequence.  Fewer than a workgroup a CU: one a chunk
    // and a joining pass (three times the state traffic, but no walk).
    if (groups >= 256 || c.T <= 7 * kQ || chunks >= kMaxUnits) {
        scan_walk_kernel<T, N, false><<<dim3(static_cast<unsigned>(2 * groups)), 256, 0, s>>>(p, dy, a.S0, a.dST, S, dS, decays, a.dS0);
    } else {
        const unsigned join = static_cast<unsigned>((static_cast<int64_t>(c.B) * c.H * (c.d_k * c.d_v / 4) + 255) / 256);
        scan_walk_kernel<T, N, true><<<dim3(static_cast<unsigned>(2 * chunks)), 256, 0, s>>>(p, dy, nullptr, nullptr, S, dS, decays, nullptr);
        walk_join_kernel<<<dim3(join, 2), 256, 0, s>>>(p, a.S0, a.dST, S, dS, decays, a.dS0);
    }
    const int slices = grad_slices(c, packed);
    float* dbp = slices > 1 ? reinterpret_cast<float*>(a.ws + w.dbp) : nullptr;
    float* dcp = slices > 1 ? reinterpret_cast<float*>(a.ws + w.dcp) : nullptr;
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&scan_grad_kernel<T, N>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(GradLds<T, N>)));
    if (e != hipSuccess) return e;
    scan_grad_kernel<T, N><<<dim3(static_cast<unsigned>(slots * c.G * slices)), 512, sizeof(GradLds<T, N>), s>>>(
        p, dy, S, dS, a.dx, a.db, a.dc, dbp, dcp, decays, sums, slices, rows);
    rates_kernel<<<dim3(units), 256, 0, s>>>(p, decays, sums, a.ddt, hp, static_cast<uint32_t>(slots));
    if (slices > 1) {
        const int64_t items = rows * (c.G * c.d_k / 4);
        join_slices_kernel<T><<<dim3(static_cast<unsigned>((items + 255) / 256)), 256, 0, s>>>(
            p, dbp, dcp, static_cast<T*>(a.db), static_cast<T*>(a.dc), slices, rows);
    }
    if (packed)
        clear_outside_kernel<T><<<dim3(static_cast<unsigned>((c.T + 255) / 256)), 256, 0, s>>>(p, static_cast<T*>(a.dx), a.ddt,
                                                                                static_cast<T*>(a.db), static_cast<T*>(a.dc));
    head_sums_kernel<<<dim3(3 * c.H), 256, 0, s>>>(p, hp, slots, a.dA, a.dD, a.dbias);
    return hipGetLastError();
}

}  // namespace

size_t scan_bwd_workspace(const la_scan_config& c, bool packed) { return bwd_ws(c, packed).total; }
int64_t scan_bwd_slots(const la_scan_config& c, bool packed) { return slot_count(c, packed); }

hipError_t launch_scan_bwd(const la_scan_config& c, const ScanArgs& a, hipStream_t s) {
    if (c.B == 0 || c.T == 0 || c.H == 0) {
        // Nothing to sum: zeros, also for the tokens of a packing without sequences and for the
        // groups of no heads; the state's gradient passes through.
        const ScanP p = scan_params(c, a);
        const int64_t rows = a.cu ? c.T : static_cast<int64_t>(c.B) * c.T;
        for (const hipError_t e : {launch_zero_rows(a.dx, c.x_dtype, rows, static_cast<int64_t>(c.H) * c.d_v, p.ld_x, s),
                                   launch_zero_rows(a.ddt, c.dt_dtype, rows, c.H, p.ld_dt, s),
                                   launch_zero_rows(a.db, c.x_dtype, rows, static_cast<int64_t>(c.G) * c.d_k, p.ld_b, s),
                                   launch_zero_rows(a.dc, c.x_dtype, rows, static_cast<int64_t>(c.G) * c.d_k, p.ld_c, s)})
            if (e != hipSuccess) return e;
        for (float* o : {a.dA, a.dD, a.dbias})
            if (o && c.H > 0) copy_or_zero_kernel<<<dim3((c.H + 255) / 256), 256, 0, s>>>(nullptr, o, c.H);
        const int64_t n = static_cast<int64_t>(c.B) * c.H * c.d_k * c.d_v;
        if (a.dS0 && n > 0) copy_or_zero_kernel<<<dim3(static_cast<unsigned>(n < 65536 * 256 ? (n + 255) / 256 : 65536)), 256, 0, s>>>(a.dST, a.dS0, n);
        return hipGetLastError();
    }
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
