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

template <class E>
struct Mfma;
template <>
struct Mfma<int8_t> {
    typedef iv4 Acc;
    static __device__ __forceinline__ Acc mul(uv4 a, uv4 b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(iv4, a), __builtin_bit_cast(iv4, b), c, 0, 0, 0);
    }
};
template <>
struct Mfma<_Float16> {
    typedef fv4 Acc;
    static __device__ __forceinline__ Acc mul(uv4 a, uv4 b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(hv8, a), __builtin_bit_cast(hv8, b), c, 0, 0, 0);
    }
};

// Row of a 32-row slab of P that lane r of 16 holds in tile b of the slab's two: a lane's results in
// the two tiles are then 8 consecutive columns of out, 8 (lane / 16) .. + 7 of the slab.
__device__ __forceinline__ int slab_row(int r, int b) { return 8 * (r >> 2) + 4 * b + (r & 3); }

// Results of TI x TJ tiles of 16 x 16 of a wave, whose first row of P is i0 and of Q j0.
template <class O, bool BITS, int TI, int TJ, class Acc>
__device__ __forceinline__ void store_tiles(const GemmArgs& a, int i0, int j0, const Acc (&acc)[TI][TJ]) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    float rs[TJ];
#pragma unroll
    for (int tj = 0; tj < TJ; tj++) {
        const int j = j0 + 16 * tj + r;
        if constexpr (BITS) rs[tj] = j < a.J ? scale_back(static_cast<const uint32_t*>(a.row)[j]) : 0.0f;
        else rs[tj] = j < a.J ? static_cast<const float*>(a.row)[j] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < TI / 2; u++) {
        const int i = i0 + 32 * u + 8 * q;
        const bool whole = a.wide && i + 8 <= a.I;
        float cs[8], bias[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const bool in = i + e < a.I;
            cs[e] = a.col && in ? a.col[i + e] : 1.0f;
            bias[e] = a.bias && in ? load_elem(a.bias, i + e, a.bias_dtype) : 0.0f;
        }
#pragma unroll
        for (int tj = 0; tj < TJ; tj++) {
            const int j = j0 + 16 * tj + r;
            if (j >= a.J) continue;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                v[e] = static_cast<float>(acc[2 * u + (e >> 2)][tj][e & 3]) * rs[tj];
                if (a.col) v[e] *= cs[e];
                if (a.bias) v[e] += bias[e];
            }
            O* o = static_cast<O*>(a.out) + static_cast<int64_t>(j) * a.ldo + i;
            if (whole) {
                if constexpr (sizeof(O) == 2) {
                    store16(o, narrow(v));
                } else {
                    store16(o, uv4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
                    store16(o + 4, uv4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (i + e < a.I) store_elem(o, e, sizeof(O) == 2 ? LA_BF16 : LA_F32, v[e]);
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

// A wave's 32 x 32 results, operands from memory straight into registers.
template <class E, class O, bool BITS>
__global__ __launch_bounds__(256) void gemm_direct_kernel(GemmArgs a) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int across = (a.I + 63) / 64;
    const int i0 = (blockIdx.x % across) * 64 + (wave & 1) * 32, j0 = (blockIdx.x / across) * 64 + (wave >> 1) * 32;
    if (i0 >= a.I || j0 >= a.J) return;
    const int ni = a.I - i0 < 32 ? a.I - i0 : 32, nj = a.J - j0 < 32 ? a.J - j0 : 32;
    const int steps = ((a.kbytes + 127) >> 7) << a.shift;
    const auto P = make_rsrc(a.P + i0 * a.ldP, (ni - 1) * a.ldP + a.kbytes);
    const auto Q = make_rsrc(a.Q + j0 * a.ldQ, (nj - 1) * a.ldQ + (static_cast<int64_t>(a.kbytes) << a.shift));
    uint32_t po[2], qo[2];
#pragma unroll
    for (int b = 0; b < 2; b++) {
        po[b] = slab_row(r, b) * static_cast<uint32_t>(a.ldP) + 16 * q;
        qo[b] = (16 * b + r) * static_cast<uint32_t>(a.ldQ) + 16 * q;
    }
    typename Mfma<E>::Acc acc[2][2] = {};
    for (int t = 0; t < steps; t++) {
        const int pk = (t >> a.shift) * 128, qk = t * 128;
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const bool in = pk + 64 * half + 16 * q < a.kbytes;  // past the row's end both operands are zero
            uv4 p[2], x[2];
#pragma unroll
            for (int b = 0; b < 2; b++) {
                p[b] = __builtin_bit_cast(uv4, __builtin_amdgcn_raw_buffer_load_b128(P, in ? po[b] + 64 * half : kOutside, pk, 0));
                x[b] = __builtin_bit_cast(uv4, __builtin_amdgcn_raw_buffer_load_b128(Q, in ? qo[b] + 64 * half : kOutside, qk, 0));
            }
#pragma unroll
            for (int ti = 0; ti < 2; ti++)
#pragma unroll
                for (int tj = 0; tj < 2; tj++) acc[ti][tj] = Mfma<E>::mul(p[ti], x[tj], acc[ti][tj]);
        }
    }
    store_tiles<O, BITS, 2, 2>(a, i0, j0, acc);
}

// LDS offset of 16-byte piece `c` of 8 in row `row` of a tile with 128 bytes of each row: the piece is
// exchanged by XOR with a number of the row, so that the 16 rows a wave reads at once lie in different
// banks.  P's rows are read in slab_row order, Q's in their own.
__device__ __forceinline__ int swizzle_p(int row) { return (row & 3) | ((row >> 1) & 4); }
__device__ __forceinline__ int swizzle_q(int row) { return row & 7; }

// 16 bytes a lane from memory to LDS, at `lds` + 16 lane.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t offset, uint32_t base) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, offset, base, 0, 0);
}

// 32 TI x 32 TJ results of a workgroup of four waves (2 x 2).  Two tiles of 128 bytes of every row in LDS:
// while the waves multiply one, the next but one's loads go straight to LDS.  A tile is two halves of 64
// bytes (one matrix instruction's depth): a half's operands are read from LDS while the half before is
// multiplied, and once a tile's second half is in registers one barrier frees its LDS.
template <class E, class O, bool BITS, int TI, int TJ, int MINW>
__global__ __launch_bounds__(256, MINW) void gemm_tile_kernel(GemmArgs a, int across, int down) {
    constexpr int BI = 32 * TI, BJ = 32 * TJ, STAGE = (BI + BJ) * 128;
    __shared__ __align__(128) char lds[2 * STAGE];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int tile = xcd_tile(blockIdx.x, across * down);
    const TileAt at = tile_order(tile, across, down);
    const int i0 = at.i * BI, j0 = at.j * BJ;
    const int ni = a.I - i0 < BI ? a.I - i0 : BI, nj = a.J - j0 < BJ ? a.J - j0 : BJ;
    const int steps = ((a.kbytes + 127) >> 7) << a.shift;
    const auto P = make_rsrc(a.P + i0 * a.ldP, (ni - 1) * a.ldP + a.kbytes);
    const auto Q = make_rsrc(a.Q + j0 * a.ldQ, (nj - 1) * a.ldQ + (static_cast<int64_t>(a.kbytes) << a.shift));
    // a wave loads 8 rows of 128 bytes at a time: rows 8 wave + 32 k + lane / 8; the piece that belongs at
    // lane % 8 of the LDS row
    const int lrow = 8 * wave + (lane >> 3);
    uint32_t po[TI], qo[TJ];
    int pc[2];
#pragma unroll
    for (int k = 0; k < TI; k++) po[k] = (lrow + 32 * k) * static_cast<uint32_t>(a.ldP) + 16 * ((lane & 7) ^ swizzle_p(lrow + 32 * k));
#pragma unroll
    for (int k = 0; k < TJ; k++) qo[k] = (lrow + 32 * k) * static_cast<uint32_t>(a.ldQ) + 16 * ((lane & 7) ^ swizzle_q(lrow + 32 * k));
    pc[0] = 16 * ((lane & 7) ^ swizzle_p(lrow)), pc[1] = 16 * ((lane & 7) ^ swizzle_q(lrow));
    auto issue = [&](int t) {
        char* s = lds + (t & 1) * STAGE + wave * 1024;
        const int pk = (t >> a.shift) * 128, qk = t * 128;
        const bool inp = pk + pc[0] < a.kbytes, inq = pk + pc[1] < a.kbytes;  // past a row's end: zero
#pragma unroll
        for (int k = 0; k < TI; k++) load_to_lds(P, s + k * 4096, inp ? po[k] : kOutside, pk);
#pragma unroll
        for (int k = 0; k < TJ; k++) load_to_lds(Q, s + BI * 128 + k * 4096, inq ? qo[k] : kOutside, qk);
    };
    const int wi = (wave & 1) * 16 * TI, wj = (wave >> 1) * 16 * TJ;
    const int prow = wi + slab_row(r, 0), qrow = wj + r;
    const int pbase = prow * 128 + 16 * (q ^ swizzle_p(prow)), qbase = BI * 128 + qrow * 128 + 16 * (q ^ swizzle_q(qrow));
    uv4 fp[2][TI], fq[2][TJ];
    auto fetch = [&](int t, int half) {  // (the second half's pieces are 4 further: bit 6 of the offset)
        const char* s = lds + (t & 1) * STAGE;
        const char* sp = s + (pbase ^ (64 * half));
        const char* sq = s + (qbase ^ (64 * half));
#pragma unroll
        for (int k = 0; k < TI; k++) fp[half][k] = *reinterpret_cast<const uv4*>(sp + (k >> 1) * 4096 + (k & 1) * 512);
#pragma unroll
        for (int k = 0; k < TJ; k++) fq[half][k] = *reinterpret_cast<const uv4*>(sq + k * 2048);
    };
    typename Mfma<E>::Acc acc[TI][TJ] = {};
    auto multiply = [&](int half) {
#pragma unroll
        for (int ti = 0; ti < TI; ti++)
#pragma unroll
            for (int tj = 0; tj < TJ; tj++) acc[ti][tj] = Mfma<E>::mul(fp[half][ti], fq[half][tj], acc[ti][tj]);
    };
    // (loads past the last tile return zero, in LDS that nobody reads again: the loop has no branches)
    issue(0);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    issue(1);
    fetch(0, 0);
    for (int t = 0; t < steps; t++) {
        fetch(t, 1);
        multiply(0);
        // tile t is in registers and tile t + 1 in LDS, in every wave
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        issue(t + 2);
        fetch(t + 1, 0);
        multiply(1);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // no load may reach LDS after the workgroup
    store_tiles<O, BITS, TI, TJ>(a, i0 + wi, j0 + wj, acc);
}

template <class E, class O, bool BITS, int TI, int TJ, int MINW>
void launch_tiles(const GemmArgs& a, hipStream_t s) {
    const int across = (a.I + 32 * TI - 1) / (32 * TI), down = (a.J + 32 * TJ - 1) / (32 * TJ);
    gemm_tile_kernel<E, O, BITS, TI, TJ, MINW><<<static_cast<unsigned>(across * down), 256, 0, s>>>(a, across, down);
}

template <class E, class O, bool BITS>
void launch_any(const GemmArgs& a, hipStream_t s) {
    const int64_t big = static_cast<int64_t>((a.I + 255) / 256) * ((a.J + 255) / 256);
    if (big >= 128) {
        launch_tiles<E, O, BITS, 8, 8, 1>(a, s);
    } else if (static_cast<int64_t>((a.I + 127) / 128) * ((a.J + 127) / 128) >= 128) {
        launch_tiles<E, O, BITS, 4, 4, 2>(a, s);
    } else {
        const unsigned grid = static_cast<unsigned>(((a.I + 63) / 64) * static_cast<int64_t>((a.J + 63) / 64));
        gemm_direct_kernel<E, O, BITS><<<grid, 256, 0, s>>>(a);
    }
}

template <class E, bool BITS>
hipError_t launch_gemm(const GemmArgs& a, int out_dtype, hipStream_t s) {
    if (out_dtype == LA_BF16) launch_any<E, uint16_t, BITS>(a, s);
    else launch_any<E, float, BITS>(a, s);
    return hipGetLastError();
}

}  // namespace la
