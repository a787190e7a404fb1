// The matrix product behind la_linear_*: out[j][i] = sum_k Q[j][k] P[i][k], both operands with the
// summed index contiguous, scales and bias in the epilogue.  8-bit integers (32-bit sums) or FP16
// (FP32 sums); a lane's 16 bytes of an operand are one matrix instruction's share in both.
#pragma once

#include "la_proj.hpp"
#include "linear_cut.hpp"

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
    int parts = 1;       // the sum is cut into this many, of part_steps x 128 bytes of Q each, part p's
    int part_steps = 0;  // result J rows below part p - 1's
    const void* row = nullptr;   // [J] or null: float factors, or the largest magnitude's bits (scale_back)
    const float* col = nullptr;  // [I] or null
    const void* bias = nullptr;  // [I] or null
    int bias_dtype = 0;
    void* out = nullptr;
    int out_dtype = LA_F32;
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
// 16 or 32 bytes of 32 different rows of out: they go through the wave's LDS (kStoreLds bytes) and leave
// as lines of 128 bytes, by 16 bytes a lane inside aligned rows, else by elements.
template <bool BITS, int TI, int TJ, class O, class Acc>
__device__ __forceinline__ void store_tiles(const GemmArgs& a, O* out, int i0, int j0, const Acc (&acc)[TI][TJ], char* lds) {
    const int lane = threadIdx.x & 63, r = lane & 31, q = lane >> 5;
    constexpr int WIDE = TI * 32 * sizeof(O) < 128 ? TI * 32 : 128 / sizeof(O);  // columns of a pass
    constexpr int LINE = WIDE * sizeof(O), PIECES = LINE / 16, ROWS = 64 / PIECES;  // rows of a store
    const bool whole = a.wide && i0 + 32 * TI <= a.I;
    float rs[TJ];
#pragma unroll
    for (int tj = 0; tj < TJ; tj++) {
        const int j = j0 + 32 * tj + r;
        if (!a.row || j >= a.J) rs[tj] = 1.0f;
        else if constexpr (BITS) rs[tj] = scale_back(static_cast<const uint32_t*>(a.row)[j]);
        else rs[tj] = static_cast<const float*>(a.row)[j];
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
                constexpr int per = sizeof(O) / 2;  // pieces of 16 bytes
                const int piece = (2 * k + q) * per, x = r & (PIECES - 1);
                char* row = lds + r * LINE;
                if constexpr (sizeof(O) == 2) {
                    *reinterpret_cast<uv4*>(row + 16 * (piece ^ x)) = narrow(v);
                } else {
                    *reinterpret_cast<fv4*>(row + 16 * (piece ^ x)) = fv4{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<fv4*>(row + 16 * ((piece + 1) ^ x)) = fv4{v[4], v[5], v[6], v[7]};
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (one wave: its own writes, in order)
            if (whole) {
#pragma unroll
                for (int n = 0; n < 32 / ROWS; n++) {
                    const int row = ROWS * n + lane / PIECES, piece = lane % PIECES, j = j0 + 32 * tj + row;
                    const uv4 v = *reinterpret_cast<const uv4*>(lds + row * LINE + 16 * (piece ^ (row & (PIECES - 1))));
                    if (j < a.J) store16(out + static_cast<int64_t>(j) * a.ldo + i0 + WIDE * pass + piece * (16 / sizeof(O)), v);
                }
            } else {
#pragma unroll
                for (int n = 0; n < WIDE / 2; n++) {
                    const int row = (64 * n + lane) / WIDE, col = (64 * n + lane) % WIDE, j = j0 + 32 * tj + row, i = i0 + WIDE * pass + col;
                    const int at = col * static_cast<int>(sizeof(O));
                    const O v = *reinterpret_cast<const O*>(lds + row * LINE + 16 * ((at >> 4) ^ (row & (PIECES - 1))) + (at & 15));
                    if (j < a.J && i < a.I) out[static_cast<int64_t>(j) * a.ldo + i] = v;
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
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

// WI x WJ waves with TI x TJ tiles of 32 x 32 each.  NS steps of 128 bytes of every row in LDS: while the
// waves multiply one, the next ones' loads go straight to LDS.  A step is four slices of one matrix
// instruction's depth: a slice's operands are read from LDS while the slice before is multiplied, and
// once a step's last slice is in registers one barrier frees its LDS for the loads of the step NS further.
// The order of reads, loads and products is spelled out (the compiler bunches the reads).  A workgroup
// takes tiles of out in turn, and the loads run on into the next one, under the stores of the one before
// (32768 x 2048 x 2048 in 8 bits: a launch of all tiles 208 us, this 192, with whole lines stored 140).
// 256 x 256 tiles are bound by power: 8192^3 in 8 bits 463 to 473 us (2320 to 2370 TOP/s) with the matrix cores 67% busy at
// 1.65 GHz, where these instructions alone, from registers, reach 3250 on the same kind of numbers.  64 x 64 ones are
// bound by LDS traffic and latency: 256 tokens, K = 2048, N = 8192 11 us, the matrix cores 9% busy.
// Of `blocks` workgroups on product a this is number `block`.  O: out's type, or void (a.out_dtype).
template <class E, class O, bool BITS, int WI, int WJ, int TI, int TJ, int NS>
__device__ __forceinline__ void gemm_units(const GemmArgs& a, int block, int blocks) {
    constexpr int NW = WI * WJ, BI = 32 * TI * WI, BJ = 32 * TJ * WJ, STAGE = (BI + BJ) * 128;
    constexpr int LI = BI / (8 * NW), LJ = BJ / (8 * NW);  // loads a wave and step: 8 rows each
    static_assert(BI % (8 * NW) == 0 && BJ % (8 * NW) == 0 && NW % 2 == 0 && (NS & (NS - 1)) == 0);
    __shared__ __align__(128) char lds[NS * STAGE + NW * kStoreLds];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 31, q = lane >> 5;
    const int across = (a.I + BI - 1) / BI, down = (a.J + BJ - 1) / BJ;
    const int tiles = across * down, units = tiles * a.parts, steps = a.part_steps;
    const int lrow = 8 * wave + (lane >> 3);  // and every 8 NW rows further: the swizzle is the same
    const int piece = 16 * ((lane & 7) ^ swizzle(lrow));
    uint32_t po[LI], qo[LJ];
#pragma unroll
    for (int k = 0; k < LI; k++) po[k] = (lrow + 8 * NW * k) * static_cast<uint32_t>(a.ldP) + piece;
#pragma unroll
    for (int k = 0; k < LJ; k++) qo[k] = (lrow + 8 * NW * k) * static_cast<uint32_t>(a.ldQ) + piece;
    // where the loads are: step `at_k` of unit `at`, a part of a tile (none left: at >= units), whose first
    // step in the whole sum is k0, and its operands' buffers
    int at = block, at_k = 0, k0 = 0;
    __amdgpu_buffer_rsrc_t P, Q;
    auto aim = [&] {
        const int unit = xcd_tile(at < units ? at : 0, units);
        const TileAt t = tile_order(unit % tiles, across, down);
        k0 = unit / tiles * steps;
        const int i0 = t.i * BI, j0 = t.j * BJ;
        const int ni = a.I - i0 < BI ? a.I - i0 : BI, nj = a.J - j0 < BJ ? a.J - j0 : BJ;
        P = make_rsrc(a.P + i0 * a.ldP, (ni - 1) * a.ldP + a.kbytes);
        Q = make_rsrc(a.Q + j0 * a.ldQ, (nj - 1) * a.ldQ + (static_cast<int64_t>(a.kbytes) << a.shift));
    };
    auto advance = [&] {
        if (++at_k >= steps) {
            at_k = 0;
            at += blocks;
            aim();
        }
    };
    // Past a row's end, and past the last tile, both operands are zero: bit 31 takes an offset outside (the
    // scalar part of the address stays inside the buffer).
    auto issue = [&](int stage) {
        char* s = lds + stage * STAGE + wave * 1024;
        int qk = (k0 + at_k) * 128, pk = ((k0 + at_k) >> a.shift) * 128;
        const uint32_t out = at < units && pk + piece < a.kbytes ? 0 : kOutside;
        if (pk >= a.kbytes) pk = qk = 0;
#pragma unroll
        for (int k = 0; k < LI; k++) load_to_lds(P, s + k * NW * 1024, po[k] | out, pk);
#pragma unroll
        for (int k = 0; k < LJ; k++) load_to_lds(Q, s + BI * 128 + k * NW * 1024, qo[k] | out, qk);
    };
    const int wi = (wave % WI) * 32 * TI, wj = (wave / WI) * 32 * TJ;
    const int prow = wi + tile_row(r), qrow = wj + r;
    const int pbase = prow * 128 + 16 * (q ^ swizzle(prow)), qbase = (BI + qrow) * 128 + 16 * (q ^ swizzle(qrow));
    uv4 fp[2][TI], fq[2][TJ];
    auto fetch = [&](int stage, int slice) {  // (the pieces of a slice are 2 further than those of the one before)
        const char* sp = lds + stage * STAGE + (pbase ^ (32 * slice));
        const char* sq = lds + stage * STAGE + (qbase ^ (32 * slice));
#pragma unroll
        for (int k = 0; k < TI; k++) fp[slice & 1][k] = *reinterpret_cast<const uv4*>(sp + k * 4096);
#pragma unroll
        for (int k = 0; k < TJ; k++) fq[slice & 1][k] = *reinterpret_cast<const uv4*>(sq + k * 4096);
    };
    typename Mfma<E>::Acc acc[TI][TJ];
    auto multiply = [&](int slice) {
#pragma unroll
        for (int ti = 0; ti < TI; ti++)
#pragma unroll
            for (int tj = 0; tj < TJ; tj++) acc[ti][tj] = Mfma<E>::mul(fp[slice & 1][ti], fq[slice & 1][tj], acc[ti][tj]);
    };
    // Pairs of loads (none, or all of a step's) with a product each, then the LDS reads among the other products.
    // (Loads to LDS keep their order with the reads behind them.)
    auto interleave = [&](auto loads) {
        constexpr int reads = TI + TJ, products = TI * TJ, with = decltype(loads)::value ? (LI + LJ) / 2 : 0;
        constexpr int rest = products > with ? products - with : 0, bunch = rest > 0 ? (reads + rest - 1) / rest : 1;
#pragma unroll
        for (int k = 0; k < with; k++) {
            __builtin_amdgcn_sched_group_barrier(0x20, 2, 0);
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        }
#pragma unroll
        for (int k = 0; k < reads; k += bunch) {
            __builtin_amdgcn_sched_group_barrier(0x100, bunch, 0);
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, products, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    aim();
#pragma unroll
    for (int k = 0; k < NS; k++) {
        if (k == 1) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
        }
        issue(k);
        advance();
    }
    fetch(0, 0);
    int stage = 0;
    int landed = 0;  // steps to come whose loads are known to have landed
    for (int id = block; id < units; id += blocks) {
#pragma unroll
        for (int k = 0; k < TI * TJ; k++) acc[k / TJ][k % TJ] = {};
        for (int t = 0; t < steps; t++) {
            const int next = (stage + 1) & (NS - 1);
#pragma unroll
            for (int k = 0; k < 3; k++) {
                fetch(stage, k + 1);
                multiply(k);
                interleave(std::false_type{});
            }
            // this step is in registers and the next one in LDS, in every wave (the ones behind it may be on their way)
            if (landed == 0) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * (LI + LJ)) : "memory");
            else landed--;
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            issue(stage);
            fetch(next, 0);
            multiply(3);
            interleave(std::true_type{});
            advance();
            stage = next;
        }
        const int unit = xcd_tile(id, units);
        const TileAt t = tile_order(unit % tiles, across, down);
        const int64_t part = unit / tiles * static_cast<int64_t>(a.J) * a.ldo;
        char* const store = lds + NS * STAGE + wave * kStoreLds;
        const int i0 = t.i * BI + wi, j0 = t.j * BJ + wj;
        if constexpr (!std::is_void_v<O>) store_tiles<BITS, TI, TJ>(a, static_cast<O*>(a.out) + part, i0, j0, acc, store);
        else if (a.out_dtype == LA_BF16) store_tiles<BITS, TI, TJ>(a, static_cast<uint16_t*>(a.out) + part, i0, j0, acc, store);
        else store_tiles<BITS, TI, TJ>(a, static_cast<float*>(a.out) + part, i0, j0, acc, store);
        landed = steps < NS - 1 ? steps : NS - 1;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // no load may reach LDS after the workgroup
}

template <class E, class O, bool BITS, int WI, int WJ, int TI, int TJ, int NS, int MINW>
__global__ __launch_bounds__(64 * WI * WJ, MINW) void gemm_tile_kernel(GemmArgs a) {
    gemm_units<E, O, BITS, WI, WJ, TI, TJ, NS>(a, blockIdx.x, gridDim.x);
}
// Two products side by side, the first one's workgroups before the second's.
template <class E, bool BITS, int WI, int WJ, int TI, int TJ, int NS, int MINW>
__global__ __launch_bounds__(64 * WI * WJ, MINW) void gemm_pair_kernel(GemmArgs a, GemmArgs b, int first) {
    const bool one = static_cast<int>(blockIdx.x) < first;
    const GemmArgs c = one ? a : b;
    gemm_units<E, void, BITS, WI, WJ, TI, TJ, NS>(c, one ? blockIdx.x : blockIdx.x - first, one ? first : gridDim.x - first);
}

template <class E, bool BITS, int WI, int WJ, int TI, int TJ, int NS, int MINW>
void launch_tiles(const GemmArgs& a, Tiling t, hipStream_t s) {
    const int64_t units = gemm_units_of(t, a.I, a.J, a.parts), most = 256 * kTilesPerCu[t];
    const unsigned grid = static_cast<unsigned>(units < most ? units : most);
    if (a.out_dtype == LA_BF16) gemm_tile_kernel<E, uint16_t, BITS, WI, WJ, TI, TJ, NS, MINW><<<grid, 64 * WI * WJ, 0, s>>>(a);
    else gemm_tile_kernel<E, float, BITS, WI, WJ, TI, TJ, NS, MINW><<<grid, 64 * WI * WJ, 0, s>>>(a);
}
template <class E, bool BITS>
hipError_t launch_gemm(const GemmArgs& a, Tiling t, hipStream_t s) {
    if (t == kTiles256) launch_tiles<E, BITS, 2, 4, 4, 2, 2, 2>(a, t, s);
    else if (t == kTiles128) launch_tiles<E, BITS, 2, 2, 2, 2, 2, 2>(a, t, s);
    else if (t == kTiles64) launch_tiles<E, BITS, 2, 2, 1, 1, 2, 4>(a, t, s);
    else launch_tiles<E, BITS, 2, 2, 1, 1, 4, 2>(a, t, s);
    return hipGetLastError();
}
// Two products in one launch, a workgroup a unit.
template <class E, bool BITS>
hipError_t launch_pair(const GemmArgs& a, const GemmArgs& b, Tiling t, hipStream_t s) {
    const int first = static_cast<int>(gemm_units_of(t, a.I, a.J, a.parts));
    const unsigned grid = static_cast<unsigned>(first + gemm_units_of(t, b.I, b.J, b.parts));
    if (t == kTiles128) gemm_pair_kernel<E, BITS, 2, 2, 2, 2, 2, 2><<<grid, 256, 0, s>>>(a, b, first);
    else if (t == kTiles64) gemm_pair_kernel<E, BITS, 2, 2, 1, 1, 2, 4><<<grid, 256, 0, s>>>(a, b, first);
    else gemm_pair_kernel<E, BITS, 2, 2, 1, 1, 4, 2><<<grid, 256, 0, s>>>(a, b, first);
    return hipGetLastError();
}

}  // namespace la
