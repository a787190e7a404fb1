// Selective scan forward: a workgroup walks the 64-token chunks of one sequence for 64 value
// columns of a head, the d_k x 64 state in its accumulators (16 columns a wave).
//
// Few heads and long sequences: the walk is cut into segments that run side by side.  A first
// pass forms each segment's own contribution to the state from zero, a small kernel joins them
// (S_in of every segment), and the full walk starts every segment from its S_in.
#include "la_scan.hpp"

namespace la {
namespace {

template <class T, int N>
struct FwdLds {
    T b[kQ * lds_row<T>(N)];
    T c[kQ * lds_row<T>(N)];
    T x[kQ * lds_row<T>(kPT)];
    T m[Mat<T>::template parts<2>][kQ * lds_row<T>(kQ)];
    Decay d;
};

// The ten 16 x 16 tiles (t, s) with s <= t, dealt to the four waves: 3, 3, 2, 2.
__device__ __forceinline__ void lower_tile(int k, int& ti, int& si) {
    ti = k < 1 ? 0 : k < 3 ? 1 : k < 6 ? 2 : 3;
    si = k - ti * (ti + 1) / 2;
}

// FULL: outputs and S_T, from the segment's S_in (or S0).  Otherwise the segment's state from
// zero into `local` and its decay into `decay`.
template <class T, int N, bool FULL>
__global__ __launch_bounds__(256) void scan_fwd_kernel(ScanP p, const float* S0, const float* Sin, void* y, float* ST,
                                                       float* local, float* decay, int nseg, int segs) {
    using MT = Mat<T>;
    constexpr int P2 = MT::template parts<2>, P3 = MT::template parts<3>;
    constexpr int RB = lds_row<T>(N), RX = lds_row<T>(kPT), RM = lds_row<T>(kQ);
    constexpr int KS = N / 32;  // contraction steps over the state's rows
    __shared__ __align__(16) FwdLds<T, N> lds;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lm = lane & 15, g = lane >> 4;

    const int tiles = p.dv / kPT;
    int64_t u = die_unit(blockIdx.x, gridDim.x);
    const int tile = static_cast<int>(u % tiles);
    u /= tiles;
    const int h = static_cast<int>(u % p.H);
    u /= p.H;
    const int seg = static_cast<int>(u % segs);  // segs: segments of this launch
    const int bi = static_cast<int>(u / segs);
    const int grp = h / (p.H / p.G);

    const SeqRange sr = seq_range(p, bi);
    const int nch = (sr.len + kQ - 1) / kQ;
    const int cps = (nch + nseg - 1) / nseg;
    const int c0 = seg * cps;
    const int c1 = c0 + cps < nch ? c0 + cps : nch;
    if (c0 >= nch && !(nch == 0 && seg == 0)) return;

    const int pcol = tile * kPT + 16 * wave + lm;  // this lane's state column
    f4 S[N / 16];
    const size_t unit = (static_cast<size_t>(bi) * p.H + h) * p.dk * p.dv;
    const float* init = nullptr;
    if (FULL) init = nseg > 1 && nch > 0 ? Sin + ((static_cast<size_t>(bi) * nseg + seg) * p.H + h) * p.dk * p.dv
                                         : (S0 ? S0 + unit : nullptr);
#pragma unroll
    for (int i = 0; i < N / 16; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int n = 16 * i + 4 * g + r;
            S[i][r] = init && n < p.dk ? init[static_cast<size_t>(n) * p.dv + pcol] : 0.0f;
        }

    const T* xg = static_cast<const T*>(p.x) + static_cast<int64_t>(h) * p.dv + tile * kPT;
    const T* bg = static_cast<const T*>(p.b) + static_cast<int64_t>(grp) * p.dk;
    const T* cg = static_cast<const T*>(p.c) + static_cast<int64_t>(grp) * p.dk;
    const float A = p.A ? p.A[h] : 0.0f;  // (no tokens: A may be missing)
    const float Dh = FULL && p.D ? p.D[h] : 0.0f;
    double cum_seg = 0.0;

    if (FULL) {  // the tiles above the diagonal that the products below read stay zero
        for (int i = threadIdx.x; i < P2 * kQ * RM; i += 256) (&lds.m[0][0])[i] = T{};
    }
    Tile<T, N, 256> tb, tc;
    Tile<T, kPT, 256> tx;
    float raw = 0.0f;
    auto fetch = [&](int ch) {
        const int64_t row0 = sr.begin + static_cast<int64_t>(ch) * kQ;
        const int live = sr.len - ch * kQ;
        tb.load(bg + row0 * p.ld_b, p.ld_b, live, p.dk);
        if (FULL) tc.load(cg + row0 * p.ld_c, p.ld_c, live, p.dk);
        tx.load(xg + row0 * p.ld_x, p.ld_x, live, kPT);
        if (wave == 0 && lane < live) raw = raw_dt(p, row0 + lane, h);
    };
    if (c0 < c1) fetch(c0);
    for (int ch = c0; ch < c1; ch++) {
        const int live = sr.len - ch * kQ;
        tb.store(lds.b, RB);
        if (FULL) tc.store(lds.c, RB);
        tx.store(lds.x, RX);
        if (wave == 0) cum_seg += make_decay(lds.d, lane < live ? step_of(p, raw, h) : 0.0f, A);
        __syncthreads();
        if (ch + 1 < c1) fetch(ch + 1);

        typename MT::Frag xT[2];  // x^T: column 16 wave + lm, tokens 32 k + 8 g ..
#pragma unroll
        for (int k = 0; k < 2; k++) xT[k] = MT::col8(lds.x, RX, 32 * k, 16 * wave, lane);

        if constexpr (FULL) {
            // M^T tiles: rows s, columns t; lane: t = lm, four consecutive s
            for (int k = wave; k < 10; k += 4) {
                int ti, si;
                lower_tile(k, ti, si);
                f4 acc = {};
#pragma unroll
                for (int ks = 0; ks < KS; ks++)
                    acc = MT::mma(MT::row8(lds.b + (16 * si + lm) * RB + 32 * ks + 8 * g),
                                  MT::row8(lds.c + (16 * ti + lm) * RB + 32 * ks + 8 * g), acc);
                const int t = 16 * ti + lm, s0 = 16 * si + 4 * g;
                const float thi = lds.d.hi[t], tlo = lds.d.lo[t];
                float m[4];
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int s = s0 + r;
                    m[r] = s <= t ? acc[r] * (pair_decay(thi, tlo, lds.d.hi[s], lds.d.lo[s]) * lds.d.delta[s]) : 0.0f;
                }
                MT::template put4<P2>(&lds.m[0][t * RM + s0], kQ * RM, m);
            }
            __syncthreads();
            typename MT::Frag Sp[KS][P2];
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
                const float v[8] = {S[2 * ks][0], S[2 * ks][1], S[2 * ks][2], S[2 * ks][3],
                                    S[2 * ks + 1][0], S[2 * ks + 1][1], S[2 * ks + 1][2], S[2 * ks + 1][3]};
                MT::template split<P2>(v, Sp[ks]);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {  // y^T: rows: columns 16 wave + 4 g + r of x; column: t
                const int t = 16 * i + lm;
                f4 acc = {};
#pragma unroll
                for (int ks = 0; ks < KS; ks++) {
                    const typename MT::Frag cf = MT::row44(lds.c + t * RB + 32 * ks + 4 * g);
#pragma unroll
                    for (int k = 0; k < P2; k++) acc = MT::mma(Sp[ks][k], cf, acc);
                }
                acc *= lds.d.head[t];
#pragma unroll
                for (int ks = 0; ks <= i / 2; ks++)
#pragma unroll
                    for (int k = 0; k < P2; k++)
                        acc = MT::mma(xT[ks], MT::row8(&lds.m[k][t * RM + 32 * ks + 8 * g]), acc);
                float xv[4];
                MT::get4(lds.x + t * RX + 16 * wave + 4 * g, xv);
#pragma unroll
                for (int r = 0; r < 4; r++) acc[r] = __builtin_fmaf(Dh, xv[r], acc[r]);
                if (t < live) {
                    const size_t at = (static_cast<size_t>(sr.begin + ch * static_cast<int64_t>(kQ) + t) * p.H + h) * p.dv +
                                      tile * kPT + 16 * wave + 4 * g;
                    if (p.out_dtype == LA_BF16)
                        *reinterpret_cast<uv2*>(static_cast<uint16_t*>(y) + at) = uv2{pack16(acc[0], acc[1]), pack16(acc[2], acc[3])};
                    else
                        *reinterpret_cast<f4*>(static_cast<float*>(y) + at) = acc;
                }
            }
        }
        // S = total S + B^T (W x)
        typename MT::Frag wx[2][P3];
#pragma unroll
        for (int k = 0; k < 2; k++) {
            float v[8];
            MT::widen8(xT[k], v);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] *= lds.d.tail[32 * k + 8 * g + j] * lds.d.delta[32 * k + 8 * g + j];
            MT::template split<P3>(v, wx[k]);
        }
        const float total = lds.d.total;
#pragma unroll
        for (int i = 0; i < N / 16; i++) {
            S[i] *= total;
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const typename MT::Frag bf = MT::col8(lds.b, RB, 32 * k, 16 * i, lane);
#pragma unroll
                for (int q = 0; q < P3; q++) S[i] = MT::mma(bf, wx[k][q], S[i]);
            }
        }
        __syncthreads();
    }
    float* out = nullptr;
    if (FULL) out = c1 == nch && ST ? ST + unit : nullptr;
    else out = local + ((static_cast<size_t>(bi) * nseg + seg) * p.H + h) * p.dk * p.dv;
    if (!FULL && threadIdx.x == 0 && tile == 0)
        decay[(static_cast<size_t>(bi) * nseg + seg) * p.H + h] = static_cast<float>(exp2(cum_seg));
    if (!out) return;
#pragma unroll
    for (int i = 0; i < N / 16; i++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int n = 16 * i + 4 * g + r;
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
    if (nseg > 1) {
        scan_fwd_kernel<T, N, false><<<dim3(static_cast<unsigned>(groups * (nseg - 1))), 256, 0, s>>>(
            p, nullptr, nullptr, nullptr, nullptr, local, decay, nseg, nseg - 1);
        const int64_t items = static_cast<int64_t>(c.B) * c.H * (c.d_k * c.d_v / 4);
        scan_join_kernel<<<dim3(static_cast<unsigned>((items + 255) / 256)), 256, 0, s>>>(p, a.S0, local, decay, nseg);
    }
    scan_fwd_kernel<T, N, true><<<dim3(static_cast<unsigned>(groups * nseg)), 256, 0, s>>>(
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
