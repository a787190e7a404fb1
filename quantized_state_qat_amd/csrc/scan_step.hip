// One token of the selective scan for a serving batch: S <- exp(Delta A) S + Delta b x^T in
// place, y = S^T c + D x.
//
// Every state element is read and written once (8 N P bytes a head against 6 N P operations):
// memory bound, the state's 16-byte accesses all issued before the first is used and passing the
// caches by (256 sequences of 16 heads, 128 x 128, in shuffled slots: 110 us, 4.9 TB/s; through them
// 15% more).  A workgroup
// owns COLS columns of one head; a lane holds 4 columns of N COLS / 1024 rows, and y's sum over
// rows is joined over the wave by lane exchanges and over the four waves in LDS.
#include "la_layer.hpp"

namespace la {
namespace {

struct StepParams {
    int B, H, G, d_v, softplus, x_dtype, dt_dtype, out_dtype, n_slots;
    int64_t ld_x, ld_b, ld_c, ld_dt;
    const void* x;
    const void* dt;
    const float* A;
    const void* b;
    const void* c;
    const float* D;
    const float* bias;
    float* S;
    const int32_t* slots;
    void* y;
};

template <int N, int COLS>
__global__ __launch_bounds__(256) void scan_step_kernel(StepParams p) {
    constexpr int CL = COLS / 4;        // lanes across the columns
    constexpr int RG = 256 / CL;        // row groups
    constexpr int R = N / RG > 0 ? N / RG : 1;
    __shared__ float red[4][COLS];
    const int tiles = p.d_v / COLS;
    const int tile = blockIdx.x % tiles;
    const int h = (blockIdx.x / tiles) % p.H;
    const int bi = blockIdx.x / (tiles * p.H);
    const int q = threadIdx.x % CL, rg = threadIdx.x / CL;
    const int col = tile * COLS + 4 * q;
    const size_t yo = (static_cast<size_t>(bi) * p.H + h) * p.d_v;
    const int slot = p.slots ? p.slots[bi] : bi;
    if (p.slots && (slot <= 0 || slot >= p.n_slots)) {  // padding
        if (threadIdx.x < COLS) store_elem(p.y, yo + tile * COLS + threadIdx.x, p.out_dtype, 0.0f);
        return;
    }
    const bool live = rg < N;  // N below the row groups: the rest only joins the sums
    float* S = p.S + (static_cast<size_t>(slot) * p.H + h) * N * p.d_v + col;
    fv4 s[R];
    if (live) {
#pragma unroll
        for (int r = 0; r < R; r++) s[r] = __builtin_nontemporal_load(reinterpret_cast<const fv4*>(S + static_cast<size_t>(rg + r * RG) * p.d_v));
    }
    const int g = h / (p.H / p.G);
    float xv[4], bv[R], cv[R];
#pragma unroll
    for (int e = 0; e < 4; e++) xv[e] = load_elem(p.x, bi * p.ld_x + static_cast<int64_t>(h) * p.d_v + col + e, p.x_dtype);
    if (live) {
#pragma unroll
        for (int r = 0; r < R; r++) {
            bv[r] = load_elem(p.b, bi * p.ld_b + g * N + rg + r * RG, p.x_dtype);
            cv[r] = load_elem(p.c, bi * p.ld_c + g * N + rg + r * RG, p.x_dtype);
        }
    }
    float d = load_elem(p.dt, bi * p.ld_dt + h, p.dt_dtype) + (p.bias ? p.bias[h] : 0.0f);
    if (p.softplus) d = fmaxf(d, 0.0f) + log1pf(expf(-fabsf(d)));
    const float a = expf(d * p.A[h]);
    float y[4] = {};
    if (live) {
#pragma unroll
        for (int r = 0; r < R; r++) {
            const float db = d * bv[r];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                s[r][e] = __builtin_fmaf(a, s[r][e], db * xv[e]);
                y[e] = __builtin_fmaf(s[r][e], cv[r], y[e]);
            }
            __builtin_nontemporal_store(s[r], reinterpret_cast<fv4*>(S + static_cast<size_t>(rg + r * RG) * p.d_v));
        }
    }
#pragma unroll
    for (int e = 0; e < 4; e++) {
        if constexpr (CL == 8) y[e] += dpp<kDppMirror>(dpp<kDppHalfMirror>(y[e]));  // lane ^ 8
        if constexpr (CL <= 16) {
            const Pair w = swap16(y[e]);
            y[e] = w.a + w.b;
        }
        const Pair w = swap32(y[e]);
        y[e] = w.a + w.b;
    }
    const int lane = threadIdx.x & 63;
    if (lane < CL) {
#pragma unroll
        for (int e = 0; e < 4; e++) red[threadIdx.x >> 6][4 * q + e] = y[e];
    }
    __syncthreads();
    if (threadIdx.x < COLS) {
        const int cc = tile * COLS + threadIdx.x;
        float o = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
        if (p.D) o = __builtin_fmaf(p.D[h], load_elem(p.x, bi * p.ld_x + static_cast<int64_t>(h) * p.d_v + cc, p.x_dtype), o);
        store_elem(p.y, yo + cc, p.out_dtype, o);
    }
}

template <int N>
hipError_t launch(const StepParams& p, hipStream_t s) {
    const int64_t heads = static_cast<int64_t>(p.B) * p.H;
    // 64 columns a workgroup (256-byte pieces of the rows), 32 for small batches, where that
    // makes workgroups for every CU (4 conversations of 16 heads: 128 -> 256 of them)
    if (heads * (p.d_v / 64) >= 512)
        scan_step_kernel<N, 64><<<static_cast<unsigned>(heads * (p.d_v / 64)), 256, 0, s>>>(p);
    else
        scan_step_kernel<N, 32><<<static_cast<unsigned>(heads * (p.d_v / 32)), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_step(const la_scan_config& c, const ScanArgs& a, hipStream_t s) {
    const StepParams p{c.B, c.H, c.G, c.d_v, c.softplus, c.x_dtype, c.dt_dtype, c.out_dtype, a.n_slots,
                       c.ld_x ? c.ld_x : static_cast<int64_t>(c.H) * c.d_v,
                       c.ld_b ? c.ld_b : static_cast<int64_t>(c.G) * c.d_k,
                       c.ld_c ? c.ld_c : static_cast<int64_t>(c.G) * c.d_k, c.ld_dt ? c.ld_dt : c.H,
                       a.x, a.dt, a.A, a.b, a.c, a.D, a.bias, a.S, a.slots, a.y};
    switch (c.d_k) {
        case 16: return launch<16>(p, s);
        case 32: return launch<32>(p, s);
        case 64: return launch<64>(p, s);
        default: return launch<128>(p, s);
    }
}

}  // namespace la
