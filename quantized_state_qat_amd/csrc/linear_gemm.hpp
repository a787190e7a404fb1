// The matrix product behind la_linear_*: out[j][i] = sum_k Q[j][k] P[i][k], both operands with the
// summed index contiguous, scales and bias in the epilogue.  8-bit integers (32-bit sums) or FP16
// (FP32 sums); a lane's 16 bytes of an operand are one matrix instruction's share in both.
#pragma once

#include "la_proj.hpp"

namespace la {

typedef int iv4 __attribute__((ext_vector_type(4)));
typedef _Float16 hv8 __attribute__((ext_vector_type(8)));

// The largest magnitude of a row's finite values scales the row by the power of two that takes it into
// [2^14, 2^15): FP16's range holds what is 2^-29 of it or larger with all its 11 bits.
__device__ __forceinline__ uint32_t up_exponent(uint32_t max_bits) {
    if (max_bits == 0) return 127;
    const uint32_t e = 268 - (max_bits >> 23);
    return e < 253 ? e : 253;
}
__device__ __forceinline__ float scale_up(uint32_t max_bits) { return __uint_as_float(up_exponent(max_bits) << 23); }
__device__ __forceinline__ float scale_back(uint32_t max_bits) { return __uint_as_float((254 - up_exponent(max_bits)) << 23); }

struct GemmArgs {
    const char* P = nullptr;  // I rows
    const char* Q = nullptr;  // J rows
    int64_t ldP = 0, ldQ = 0;  // bytes between rows, multiples of 16
    int I = 0, J = 0;
    int kbytes = 0;  // bytes of a row of P that are summed, a multiple of 16
    int shift = 0;   // Q holds 1 << shift parts of each 128 bytes of P, beside each other
    const void* row = nullptr;   // [J]: float factors, or the largest magnitude's bits (scale_back)
    const float* col = nullptr;  // [I] or null
    const void* bias = nullptr;  // [I] or null
    int bias_dtype = 0;
    void* out = nullptr;
    int64_t ldo = 0;  // elements
    int wide = 0;     // rows of out are 16-byte aligned
};

typedef int iv16 __attribute__((ext_vector_type(16)));
typedef float fv16 __attribute__((ext_vector_type(16)));

// One matrix instruction: 32 x 32 results, 32 bytes of the summed index; lane l holds 16 of them,
// 16 (l / 32) .. + 15, of row l % 32 of each operand.  (16 x 16 results over 64 bytes read the same LDS
// for the same work in twice the instructions: 8192^3 in 8 bits 1975 against 2140 TOP/s, four waves.)
template <class E>
struct Mfma;
template <>
struct Mfma<int8_t> {
    typedef iv16 Acc;
    static __device__ __forceinline__ Acc mul(uv4 a, uv4 b, Acc c) {
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(iv4, a), __builtin_bit_cast(iv4, b), c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16> {
    typedef fv16 Acc;
    static __device__ __forceinline__ Acc mul(uv4 a, uv4 b, Acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hv8, a), __builtin_bit_cast(hv8, b), c, 0, 0, 0);
    }
};

// Row of a tile's 32 rows of P that lane r of 32 holds: results v of lane l are then columns
// 16 (v / 8) + 8 (l / 32) + v % 8 of the tile (row 8 (v / 4) + 4 (l / 32) + v % 4 of the instruction is
// result v of a lane).
__device__ __forceinline__ int tile_row(int r) { return 16 * (r >> 4) + 8 * ((r >> 2) & 1) + 4 * ((r >> 3) & 1) + (r & 3); }

__device__ __forceinline__ void load_eight(const float* p, float (&v)[8]) {
    float a[4], b[4];
    widen(load16(p), a);
    widen(load16(p + 4), b);
#pragma unroll
    for (int e = 0; e < 4; e++) {
        v[e] = a[e];
        v[4 + e] = b[e];
    }
}

// 128 bytes of 32 rows of out, on their way from a wave's registers to whole lines of memory.
constexpr int kStoreLds = 4096;

// Results of a wave's TI x TJ tiles, the first one's at column i0 and row j0 of out.  A lane's results are
// 16 or 32 bytes of 32 different rows of out; where the tile lies inside, they go through the wave's LDS
// (kStoreLds bytes) and leave as lines of 128 bytes.
template <class O, bool BITS, int TI, int TJ, class Acc>
__device__ __forceinline__ void store_tiles(const GemmArgs& a, int i0, int j0, const Acc (&acc)[TI][TJ], char* lds) {
    const int lane = threadIdx.x & 63, r = lane & 31, q = lane >> 5;
    constexpr int WIDE = TI * 32 * sizeof(O) < 128 ? TI * 32 : 128 / sizeof(O);  // columns of a pass
    constexpr int LINE = WIDE * sizeof(O), PIECES = LINE / 16, ROWS = 64 / PIECES;  // rows of a store
    const bool whole = a.wide && i0 + 32 * TI <= a.I;
    float rs[TJ];
#pragma unroll
    for (int tj = 0; tj < TJ; tj++) {
        const int j = j0 + 32 * tj + r;
        if constexpr (BITS) rs[tj] = j < a.J ? scale_back(static_cast<const uint32_t*>(a.row)[j]) : 0.0f;
        else rs[tj] = j < a.J ? static_cast<const float*>(a.row)[j] : 0.0f;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (the kernel counts on it: every load before has landed)
#pragma unroll
    for (int pass = 0; pass < TI * 32 / WIDE; pass++) {
        constexpr int EIGHTS = WIDE / 16;  // eights of columns that a lane has of a pass
#pragma unroll
        for (int tj = 0; tj < TJ; tj++) {
#pragma unroll
            for (int k = 0; k < EIGHTS; k++) {
                const int at = WIDE / 16 * pass + k, i = i0 + 16 * at + 8 * q;  // sixteens of columns from i0
                float cs[8], bias[8];
                if (i + 8 <= a.I) {
                    if (a.col) load_eight(a.col + i, cs);
                    if (a.bias) {
                        if (a.bias_dtype == LA_BF16) widen(load16(static_cast<const uint16_t*>(a.bias) + i), bias);
                        else load_eight(static_cast<const float*>(a.bias) + i, bias);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const bool in = i + e < a.I;
                        cs[e] = a.col && in ? a.col[i + e] : 1.0f;
                        bias[e] = a.bias && in ? load_elem(a.bias, i + e, a.bias_dtype) : 0.0f;
                    }
                }
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    v[e] = static_cast<float>(acc[at / 2][tj][8 * (at % 2) + e]) * rs[tj];
                    if (a.col) v[e] *= cs[e];
                    if (a.bias) v[e] += bias[e];
                }
                if (whole) {
                    constexpr int per = sizeof(O) / 2;  // pieces of 16 bytes
                    const int piece = (2 * k + q) * per, x = r & (PIECES - 1);
                    char* row = lds + r * LINE;
                    if constexpr (sizeof(O) == 2) {
                        *reinterpret_cast<uv4*>(row + 16 * (piece ^ x)) = narrow(v);
                    } else {
                        *reinterpret_cast<fv4*>(row + 16 * (piece ^ x)) = fv4{v[0], v[1], v[2], v[3]};
                        *reinterpret_cast<fv4*>(row + 16 * ((piece + 1) ^ x)) = fv4{v[4], v[5], v[6], v[7]};
                    }
                } else {
                    const int j = j0 + 32 * tj + r;
                    O* o = static_cast<O*>(a.out) + static_cast<int64_t>(j) * a.ldo + i;
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (j < a.J && i + e < a.I) store_elem(o, e, sizeof(O) == 2 ? LA_BF16 : LA_F32, v[e]);
                }
            }
            if (whole) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (one wave: its own writes, in order)
#pragma unroll
                for (int n = 0; n < 32 / ROWS; n++) {
                    const int row = ROWS * n + lane / PIECES, piece = lane % PIECES, j = j0 + 32 * tj + row;
                    const uv4 v = *reinterpret_cast<const uv4*>(lds + row * LINE + 16 * (piece ^ (row & (PIECES - 1))));
                    if (j < a.J) store16(static_cast<O*>(a.out) + static_cast<int64_t>(j) * a.ldo + i0 + WIDE * pass + piece * (16 / sizeof(O)), v);
                }
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
        }
    }
}

// Workgroups go to the eight dies in turn: workgroup b works on a tile such that each die has a range of
// consecutive ones.
__device__ __forceinline__ int xcd_tile(int b, int n) {
    const int per = n / 8, more = n % 8, die = b % 8, k = b / 8;
    return die * per + (die < more ? die : more) + k;
}
// Consecutive tiles cover blocks of 8 rows of tiles, column by column: what the workgroups of a die work
// on at a time shares rows of both operands.
struct TileAt {
    int i, j;
};
__device__ __forceinline__ TileAt tile_order(int tile, int across, int down) {
    const int block = tile / (8 * across), in = tile % (8 * across);
    const int rows = down - 8 * block < 8 ? down - 8 * block : 8;
    return {in / rows, 8 * block + in % rows};
}

constexpr uint32_t kOutside = 0x80000000u;  // an offset past every operand's buffer: such loads return zero

// LDS holds 128 bytes of every row of a tile; 16-byte piece c of 8 of row `row` lies at c ^ swizzle(row),
// so that lanes that read the same piece of neighbouring rows at once reach different banks (no
// conflicts counted; with row & 7 half of the reads' cycles were).
__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }

// 16 bytes a lane from memory to LDS, at `lds` + 16 lane.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t offset, uint32_t base) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, offset, base, 0, 0);
}

// WI x WJ waves with TI x TJ tiles of 32 x 32 each.  Two tiles of 128 bytes of every row in LDS: while the
// waves multiply one, the next one's loads go straight to LDS.  A tile is two halves of 64 bytes (two
// matrix instructions deep): a half's operands are read from LDS while the half before is multiplied,
// and once a tile's second half is in registers one barrier frees its LDS for the loads of the next but
// one.  The order of the two kinds of instructions is spelled out (the compiler bunches the reads: 8192^3
// in 8 bits 2320 against 2380 TOP/s).  A workgroup takes tiles of out in turn, and the loads run on into
// the next one, under the stores of the one before.
template <class E, class O, bool BITS, int WI, int WJ, int TI, int TJ, int MINW>
__global__ __launch_bounds__(64 * WI * WJ, MINW) void gemm_tile_kernel(GemmArgs a, int across, int down) {
    constexpr int NW = WI * WJ, BI = 32 * TI * WI, BJ = 32 * TJ * WJ, STAGE = (BI + BJ) * 128;
    constexpr int LI = BI / (8 * NW), LJ = BJ / (8 * NW);  // loads a wave: 8 rows each
    static_assert(BI % (8 * NW) == 0 && BJ % (8 * NW) == 0 && NW % 2 == 0);
    __shared__ __align__(128) char lds[2 * STAGE + NW * kStoreLds];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 31, q = lane >> 5;
    const int tiles = across * down;
    const int steps = ((a.kbytes + 127) >> 7) << a.shift;
    const int lrow = 8 * wave + (lane >> 3);  // and every 8 NW rows further: the swizzle is the same
    const int piece = 16 * ((lane & 7) ^ swizzle(lrow));
    uint32_t po[LI], qo[LJ];
#pragma unroll
    for (int k = 0; k < LI; k++) po[k] = (lrow + 8 * NW * k) * static_cast<uint32_t>(a.ldP) + piece;
#pragma unroll
    for (int k = 0; k < LJ; k++) qo[k] = (lrow + 8 * NW * k) * static_cast<uint32_t>(a.ldQ) + piece;
    // where the loads are: step `at_k` of tile `at` (none left: at >= tiles), its operands' buffers
    int at = blockIdx.x, at_k = 0;
    __amdgpu_buffer_rsrc_t P, Q;
    auto aim = [&] {
        const TileAt t = tile_order(xcd_tile(at < tiles ? at : 0, tiles), across, down);
        const int i0 = t.i * BI, j0 = t.j * BJ;
        const int ni = a.I - i0 < BI ? a.I - i0 : BI, nj = a.J - j0 < BJ ? a.J - j0 : BJ;
        P = make_rsrc(a.P + i0 * a.ldP, (ni - 1) * a.ldP + a.kbytes);
        Q = make_rsrc(a.Q + j0 * a.ldQ, (nj - 1) * a.ldQ + (static_cast<int64_t>(a.kbytes) << a.shift));
    };
    auto advance = [&] {
        if (++at_k >= steps) {
            at_k = 0;
            at += gridDim.x;
            aim();
        }
    };
    // Past a row's end, and past the last tile, both operands are zero: bit 31 takes an offset outside (the
    // scalar part of the address stays inside the buffer).
    auto issue = [&](int stage) {
        char* s = lds + stage * STAGE + wave * 1024;
        const int qk = at_k * 128, pk = (at_k >> a.shift) * 128;
        const uint32_t out = at < tiles && pk + piece < a.kbytes ? 0 : kOutside;
#pragma unroll
        for (int k = 0; k < LI; k++) load_to_lds(P, s + k * NW * 1024, po[k] | out, pk);
#pragma unroll
        for (int k = 0; k < LJ; k++) load_to_lds(Q, s + BI * 128 + k * NW * 1024, qo[k] | out, qk);
    };
    const int wi = (wave % WI) * 32 * TI, wj = (wave / WI) * 32 * TJ;
    const int prow = wi + tile_row(r), qrow = wj + r;
    const int pbase = prow * 128 + 16 * (q ^ swizzle(prow)), qbase = BI * 128 + qrow * 128 + 16 * (q ^ swizzle(qrow));
    uv4 fp[2][2][TI], fq[2][2][TJ];
    auto fetch = [&](int stage, int half) {  // (the pieces of instruction h of a half are 4 half + 2 h further)
        const char* s = lds + stage * STAGE;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const char* sp = s + (pbase ^ (64 * half + 32 * h));
            const char* sq = s + (qbase ^ (64 * half + 32 * h));
#pragma unroll
            for (int k = 0; k < TI; k++) fp[half][h][k] = *reinterpret_cast<const uv4*>(sp + k * 4096);
#pragma unroll
            for (int k = 0; k < TJ; k++) fq[half][h][k] = *reinterpret_cast<const uv4*>(sq + k * 4096);
        }
    };
    typename Mfma<E>::Acc acc[TI][TJ];
    auto multiply = [&](int half) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int ti = 0; ti < TI; ti++)
#pragma unroll
                for (int tj = 0; tj < TJ; tj++) acc[ti][tj] = Mfma<E>::mul(fp[half][h][ti], fq[half][h][tj], acc[ti][tj]);
    };
    // one LDS read (and, with LOADS, a share of the loads), then a share of the products, and so on
    auto interleave = [&](auto loads) {
        constexpr int reads = 2 * (TI + TJ), products = 2 * TI * TJ, share = products / reads;
#pragma unroll
        for (int k = 0; k < reads; k++) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if constexpr (decltype(loads)::value) __builtin_amdgcn_sched_group_barrier(0x20, (LI + LJ + reads - 1) / reads, 0);
            if constexpr (share > 0) __builtin_amdgcn_sched_group_barrier(0x8, share, 0);
        }
        if constexpr (products > share * reads) __builtin_amdgcn_sched_group_barrier(0x8, products - share * reads, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    aim();
    issue(0);
    advance();
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    issue(1);
    advance();
    fetch(0, 0);
    int stage = 0;
    bool landed = false;  // the loads of the next step are known to have landed
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
#pragma unroll
        for (int ti = 0; ti < TI; ti++)
#pragma unroll
            for (int tj = 0; tj < TJ; tj++) acc[ti][tj] = {};
        for (int t = 0; t < steps; t++) {
            fetch(stage, 1);
            multiply(0);
            interleave(std::false_type{});
            // this step is in registers and the next one in LDS, in every wave
            if (!landed) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            landed = false;
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            issue(stage);
            fetch(stage ^ 1, 0);
            multiply(1);
            interleave(std::true_type{});
            advance();
            stage ^= 1;
        }
        const TileAt t = tile_order(xcd_tile(tile, tiles), across, down);
        store_tiles<O, BITS, TI, TJ>(a, t.i * BI + wi, t.j * BJ + wj, acc, lds + 2 * STAGE + wave * kStoreLds);
        landed = steps > 0;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // no load may reach LDS after the workgroup
}

// PER: workgroups that a CU holds.
template <class E, class O, bool BITS, int WI, int WJ, int TI, int TJ, int MINW, int PER>
void launch_tiles(const GemmArgs& a, hipStream_t s) {
    constexpr int BI = 32 * TI * WI, BJ = 32 * TJ * WJ;
    const int across = (a.I + BI - 1) / BI, down = (a.J + BJ - 1) / BJ;
    const int tiles = across * down, most = 256 * PER;
    gemm_tile_kernel<E, O, BITS, WI, WJ, TI, TJ, MINW><<<static_cast<unsigned>(tiles < most ? tiles : most), 64 * WI * WJ, 0, s>>>(a, across, down);
}

template <class E, class O, bool BITS>
void launch_any(const GemmArgs& a, hipStream_t s) {
    const auto tiles = [&](int bi, int bj) { return static_cast<int64_t>((a.I + bi - 1) / bi) * ((a.J + bj - 1) / bj); };
    if (tiles(256, 256) >= 128) launch_tiles<E, O, BITS, 2, 4, 4, 2, 2, 1>(a, s);
    else if (tiles(128, 128) >= 128) launch_tiles<E, O, BITS, 2, 2, 2, 2, 2, 2>(a, s);
    else launch_tiles<E, O, BITS, 2, 2, 1, 1, 4, 4>(a, s);
}

template <class E, bool BITS>
hipError_t launch_gemm(const GemmArgs& a, int out_dtype, hipStream_t s) {
    if (out_dtype == LA_BF16) launch_any<E, uint16_t, BITS>(a, s);
    else launch_any<E, float, BITS>(a, s);
    return hipGetLastError();
}

}  // namespace la
