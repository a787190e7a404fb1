// Selective scan forward: a workgroup walks the 64-token chunks of one sequence for 64 value
// columns of a head, the d_k x 64 state in its accumulators.
//
// Only the state's update is serial.  Eight waves, two roles: waves 0..3 bring chunk i + 1 into
// LDS and form its M (and the decays of chunk i + 2, on the wave with one tile of M); waves
// 4..7 (16 columns each) meanwhile form chunk i's output and update the state.  Two barriers a
// chunk (staged | done) and two LDS buffers; the loads of chunk i + 3 are issued while chunk i is
// in work.  With every wave doing every part in turn a chunk took 5.3 us, most of it waiting (one
// wave a SIMD).
//
// Few heads and long sequences: the walk is cut into segments that run side by side.  A first
// pass forms each segment's own contribution to the state from zero, a small kernel joins them
// (S_in of every segment), and the full walk starts every segment from its S_in.
#include "la_scan.hpp"

namespace la {
namespace {

template <class T, int N, bool FULL>
struct FwdLds {
    T b[kQ * lds_row<T>(N)];
    T c[FULL ? kQ * lds_row<T>(N) : 8];
    T x[kQ * lds_row64<T>()];
    T m[FULL ? Mat<T>::template parts<2> : 1][FULL ? kQ * lds_row64<T>() : 8];
};
// Two buffers where they fit (160 KB; not FP32 with d_k = 128: the roles then take turns), and
// three of the decays, which are formed earlier.
template <class T, int N, bool FULL>
constexpr int kBufs = 2 * sizeof(FwdLds<T, N, FULL>) + 3 * sizeof(Decay) <= 160 * 1024 ? 2 : 1;
template <class T, int N, bool FULL>
constexpr size_t kFwdLds = kBufs<T, N, FULL> * sizeof(FwdLds<T, N, FULL>) + 3 * sizeof(Decay);

// FULL: outputs and S_T, from the segment's S_in (or S0).  Otherwise the segment's state from
// zero into `local` and its decay into `decay`.
template <class T, int N, bool FULL>
__global__ __launch_bounds__(512) void scan_fwd_kernel(ScanP p, const float* S0, const float* Sin, void* y, float* ST,
                                                       float* local, float* decay, int nseg, int segs) {
    using MT = Mat<T>;
    constexpr int P2 = MT::template parts<2>, P3 = MT::template parts<3>;
    constexpr int RB = lds_row<T>(N), RX = lds_row64<T>(), RM = lds_row64<T>();
    constexpr int KS = N / 32;  // contraction steps over the state's rows
    constexpr int NB = kBufs<T, N, FULL>;
    using Buf = FwdLds<T, N, FULL>;
    extern __shared__ __align__(16) char raw_lds[];
    Buf* const bufs = reinterpret_cast<Buf*>(raw_lds);
    Decay* const decays = reinterpret_cast<Decay*>(raw_lds + NB * sizeof(Buf));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lm = lane & 15, g = lane >> 4;

    const int tiles = p.dv / kPT;
    uint32_t u = die_unit(blockIdx.x, gridDim.x);
    const int tile = take(u, tiles), h = take(u, p.H), seg = take(u, segs);  // segs: segments of this launch
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
    const float A = p.A ? p.A[h] : 0.0f;  // (no tokens: A may be missing)
    const float Dh = FULL && p.D ? p.D[h] : 0.0f, bias = p.bias ? p.bias[h] : 0.0f;

    if (FULL) {  // the tiles above the diagonal that the products below read stay zero
        for (int q = 0; q < NB; q++)
            for (int i = threadIdx.x; i < P2 * kQ * RM; i += 512) (&bufs[q].m[0][0])[i] = T{};
        __syncthreads();
    }

    if (wave < 4) {
        // ------------------------------------------------------------ chunks into LDS, and M
        const T* xg = static_cast<const T*>(p.x) + static_cast<int64_t>(h) * p.dv + tile * kPT;
        const T* bg = static_cast<const T*>(p.b) + static_cast<int64_t>(grp) * p.dk;
        const T* cg = static_cast<const T*>(p.c) + static_cast<int64_t>(grp) * p.dk;
        struct None {};
        struct Ahead {
            Tile<T, N, 256> b;
            std::conditional_t<FULL, Tile<T, N, 256>, None> c;
            Tile<T, kPT, 256> x;
            DtAhead raw;
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
            r.x.load(xg + row0 * p.ld_x, p.ld_x, live, kPT);
            if (wave == 3) r.raw.fetch(p, row0, h, lane, live);
        };
        double cum_seg = 0.0;
        auto decays_of = [&](int ch, const Ahead& r) {  // by one wave
            cum_seg += make_decay(decays[(ch - c0) % 3], r.raw.value(p) + bias, p.softplus, sr.len - ch * kQ, A);
        };
        auto stage = [&](Buf& lds, const Ahead& r) {
            r.b.store(lds.b, RB);
            if constexpr (FULL) r.c.store(lds.c, RB);
            r.x.store(lds.x, RX);
        };
        // M^T tiles (ti, s_first ..): rows s, columns t; lane: t, four consecutive s.  D goes onto the diagonal.
        auto pair_row = [&](Buf& lds, const Decay& d, int ti, int s_first, auto count) {
            constexpr int C = decltype(count)::value;
            typename MT::Frag bf[C][KS], cf[KS];
            const int t = 16 * ti + lm;
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
                cf[ks] = MT::row8(lds.c + t * RB + 32 * ks + 8 * g);
#pragma unroll
                for (int q = 0; q < C; q++) bf[q][ks] = MT::row8(lds.b + (16 * (s_first + q) + lm) * RB + 32 * ks + 8 * g);
            }
            const float thi = d.hi[t], tlo = d.lo[t];
            f4 shi[C], slo[C], sdl[C];
#pragma unroll
            for (int q = 0; q < C; q++) {
                const int s0 = 16 * (s_first + q) + 4 * g;
                shi[q] = *reinterpret_cast<const f4*>(d.hi + s0);
                slo[q] = *reinterpret_cast<const f4*>(d.lo + s0);
                sdl[q] = *reinterpret_cast<const f4*>(d.delta + s0);
            }
            __builtin_amdgcn_sched_barrier(0);
            f4 acc[C] = {};
#pragma unroll
            for (int ks = 0; ks < KS; ks++)
#pragma unroll
                for (int q = 0; q < C; q++) acc[q] = MT::mma(bf[q][ks], cf[ks], acc[q]);
#pragma unroll
            for (int q = 0; q < C; q++) {
                const int s0 = 16 * (s_first + q) + 4 * g;
                float m[4];
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    m[r] = acc[q][r] * (pair_decay(thi, tlo, shi[q][r], slo[q][r]) * sdl[q][r]);
                    m[r] = s0 + r < t ? m[r] : s0 + r == t ? m[r] + Dh : 0.0f;
                }
                MT::template put4<P2>(&lds.m[0][t * RM + s0], kQ * RM, m);
            }
        };
        auto pairs = [&](Buf& lds, const Decay& d) {  // the ten tiles; the wave with one also forms the decays
            if constexpr (FULL) {
                using std::integral_constant;
                if (wave == 0) pair_row(lds, d, 3, 0, integral_constant<int, 3>{});
                if (wave == 1) pair_row(lds, d, 2, 0, integral_constant<int, 3>{});
                if (wave == 2) pair_row(lds, d, 1, 0, integral_constant<int, 2>{});
                if (wave == 2) pair_row(lds, d, 3, 3, integral_constant<int, 1>{});
                if (wave == 3) pair_row(lds, d, 0, 0, integral_constant<int, 1>{});
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
                    if (ch < c1) pairs(lds, decays[(ch - c0) % 3]);
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
                    pairs(bufs[0], decays[(ch - c0) % 3]);
                    __syncthreads();
                }
                __syncthreads();
            }
        }
        if (!FULL && threadIdx.x == 192 && tile == 0)
            decay[(static_cast<size_t>(bi) * nseg + seg) * p.H + h] = static_cast<float>(exp2(cum_seg));
        return;
    }

    // ---------------------------------------------------------------- outputs and the state
    const int w0 = 16 * (wave - 4);                // this wave's columns of the tile
    const int pcol = tile * kPT + w0 + lm;         // this lane's state column
    f4 S[N / 16];
    const size_t unit = (static_cast<size_t>(bi) * p.H + h) * p.dk * p.dv;
    const float* init = nullptr;
    if (FULL) init = nseg > 1 && nch > 0 ? Sin + ((static_cast<size_t>(bi) * nseg + seg) * p.H + h) * p.dk * p.dv
                                         : (S0 ? S0 + unit : nullptr);
#pragma unroll
    for (int i = 0; i < N / 16; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int n = state_n(i, 4 * g + r);
            S[i][r] = init && n < p.dk ? init[static_cast<size_t>(n) * p.dv + pcol] : 0.0f;
        }
    // LDS reads are issued together ahead of the products that take them (the fences keep the
    // compiler from sinking each to its use, where its whole latency would be waited for), and
    // products on one accumulator are kept four apart.
    //
    // What needs no state: W x, and M x as y^T (rows: columns w0 + 4 g + r of x; column: t).
    auto stateless = [&](const Buf& lds, const Decay& d, f4 (&acc)[4], typename MT::Frag (&wx)[2][P3]) {
        typename MT::Frag xT[2], mf[2][P2][4];  // x^T: column w0 + lm
        float wt[2][8];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            xT[k] = MT::col8(lds.x, RX, 32 * k, w0, lane);
            get8(d.w + 32 * k + 8 * g, wt[k]);
        }
        if constexpr (FULL) {
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
#pragma unroll
                for (int k = 0; k < P2; k++)
#pragma unroll
                    for (int i = 2 * ks; i < 4; i++) mf[ks][k][i] = MT::row8(&lds.m[k][(16 * i + lm) * RM + 32 * ks + 8 * g]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 4; i++) acc[i] = f4{};
#pragma unroll
            for (int ks = 0; ks < 2; ks++)
#pragma unroll
                for (int k = 0; k < P2; k++)
#pragma unroll
                    for (int i = 2 * ks; i < 4; i++) acc[i] = MT::mma(xT[ks], mf[ks][k][i], acc[i]);
        }
#pragma unroll
        for (int k = 0; k < 2; k++) {
            float v[8];
            MT::widen8(xT[k], v);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] *= wt[k][j];
            MT::template split<P3>(v, wx[k]);
        }
    };
    const int es = p.out_dtype == LA_BF16 ? 2 : 4;
    const int64_t ld_y = static_cast<int64_t>(p.H) * p.dv;
    constexpr int AHEAD = sizeof(T) == 2 ? KS : 1;  // contraction steps whose c rows are read together
    auto output = [&](int ch, const Buf& lds, const Decay& d, const f4 (&acc)[4]) {
        f4 y4[4] = {};
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
            for (int ks = 0; ks < AHEAD; ks++) {
                const int i0 = 2 * (k0 + ks);
                typename MT::Frag Sp[P2];
                const float v[8] = {S[i0][0], S[i0][1], S[i0][2], S[i0][3], S[i0 + 1][0], S[i0 + 1][1], S[i0 + 1][2], S[i0 + 1][3]};
                MT::template split<P2>(v, Sp);
#pragma unroll
                for (int k = 0; k < P2; k++)
#pragma unroll
                    for (int i = 0; i < 4; i++) y4[i] = MT::mma(Sp[k], cf[ks][i], y4[i]);
            }
        }
        // rows behind the sequence lie behind the buffer's end
        const int live = sr.len - ch * kQ < kQ ? sr.len - ch * kQ : kQ;
        char* row0 = static_cast<char*>(y) + ((sr.begin + ch * static_cast<int64_t>(kQ)) * ld_y + static_cast<int64_t>(h) * p.dv + tile * kPT) * es;
        const __amdgpu_buffer_rsrc_t ry = make_rsrc(row0, static_cast<size_t>(live) * ld_y * es);
#pragma unroll
        for (int i = 0; i < 4; i++) {
#pragma unroll
            for (int r = 0; r < 4; r++) y4[i][r] = __builtin_fmaf(y4[i][r], head[i], acc[i][r]);
            const int off = ((16 * i + lm) * static_cast<int>(ld_y) + w0 + 4 * g) * es;
            if (es == 2)
                __builtin_amdgcn_raw_buffer_store_b64(uv2{pack16(y4[i][0], y4[i][1]), pack16(y4[i][2], y4[i][3])}, ry, off, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uv4, y4[i]), ry, off, 0, 0);
        }
    };
    auto update = [&](const Buf& lds, const Decay& d, const typename MT::Frag (&wx)[2][P3]) {  // S = total S + B^T (W x)
        const float total = d.total[0];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            typename MT::Frag bf[N / 16];
#pragma unroll
            for (int i = 0; i < N / 16; i++) bf[i] = MT::col8_state(lds.b, RB, 32 * k, i, lane);
            __builtin_amdgcn_sched_barrier(0);
            if (k == 0) {
#pragma unroll
                for (int i = 0; i < N / 16; i++) S[i] *= total;
            }
#pragma unroll
            for (int q = 0; q < P3; q++)
#pragma unroll
                for (int i = 0; i < N / 16; i++) S[i] = MT::mma(bf[i], wx[k][q], S[i]);
        }
    };
    if constexpr (NB == 2) {
        auto step = [&](int ch, const Buf& lds) {  // beside the staging of chunk ch + 1 and its M
            const Decay& d = decays[(ch - c0 + 3) % 3];
            typename MT::Frag wx[2][P3];
            f4 acc[4];
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
            const Decay& d = decays[(ch - c0) % 3];
            typename MT::Frag wx[2][P3];
            f4 acc[4];
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
    else out = local + ((static_cast<size_t>(bi) * nseg + seg) * p.H + h) * p.dk * p.dv;
    if (!out) return;
#pragma unroll
    for (int i = 0; i < N / 16; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int n = state_n(i, 4 * g + r);
            if (n < p.dk) out[static_cast<size_t>(n) * p.dv + pcol] = S[i][r];
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
    for (int s = 0; s < nseg && s * cps < nch; s++) {
        const size_t at = (static_cast<size_t>(bi) * nseg + s) * p.H + h;
        fv4* l = reinterpret_cast<fv4*>(local) + at * per + e;
        const bool more = (s + 1) * cps < nch;  // the last segment's own state is not formed
        const fv4 own = more ? *l : fv4{};
        *l = S;
        if (more) S = S * decay[at] + own;
    }
}

// Segments of a sequence: one while the heads alone fill the chip (two workgroups a CU), else
// enough for that, of at least four chunks each: the first pass costs about half a full walk,
// so a cut pays from two to three segments on.
int segments(const la_scan_config& c) {
    const int64_t groups = static_cast<int64_t>(c.B) * c.H * (c.d_v / kPT);
    const int64_t chunks = (c.T + kQ - 1) / kQ;
    if (groups == 0) return 1;
    int64_t n = 512 / groups;
    if (n > chunks / 4) n = chunks / 4;
    return n < 3 ? 1 : static_cast<int>(n);
}

size_t local_bytes(const la_scan_config& c, int nseg) {
    return static_cast<size_t>(c.B) * nseg * c.H * c.d_k * c.d_v * sizeof(float);
}

template <class T, int N>
hipError_t launch(const la_scan_config& c, const ScanArgs& a, hipStream_t s) {
    const ScanP p = scan_params(c, a);
    const int nseg = segments(c);
    const int64_t groups = static_cast<int64_t>(c.B) * c.H * (c.d_v / kPT);
    float* local = reinterpret_cast<float*>(a.ws);
    float* decay = reinterpret_cast<float*>(a.ws + (nseg > 1 ? local_bytes(c, nseg) : 0));
    auto allow = [](auto& kernel, size_t bytes) {
        return hipFuncSetAttribute(reinterpret_cast<const void*>(&kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(bytes));
    };
    hipError_t e;
    if (nseg > 1) {
        constexpr size_t bytes = kFwdLds<T, N, false>;
        e = allow(scan_fwd_kernel<T, N, false>, bytes);
        if (e != hipSuccess) return e;
        scan_fwd_kernel<T, N, false><<<dim3(static_cast<unsigned>(groups * (nseg - 1))), 512, bytes, s>>>(
            p, nullptr, nullptr, nullptr, nullptr, local, decay, nseg, nseg - 1);
        const int64_t items = static_cast<int64_t>(c.B) * c.H * (c.d_k * c.d_v / 4);
        scan_join_kernel<<<dim3(static_cast<unsigned>((items + 255) / 256)), 256, 0, s>>>(p, a.S0, local, decay, nseg);
    }
    constexpr size_t bytes = kFwdLds<T, N, true>;
    e = allow(scan_fwd_kernel<T, N, true>, bytes);
    if (e != hipSuccess) return e;
    scan_fwd_kernel<T, N, true><<<dim3(static_cast<unsigned>(groups * nseg)), 512, bytes, s>>>(
        p, a.S0, local, a.y, a.ST, nullptr, nullptr, nseg, nseg);
    return hipGetLastError();
}

}  // namespace

size_t scan_fwd_workspace(const la_scan_config& c) {
    const int nseg = segments(c);
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
