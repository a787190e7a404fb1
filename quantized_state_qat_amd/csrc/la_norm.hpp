// Row helpers of the norms: pieces of 8 columns, sums and maxima over the lanes that hold a row, and
// the 8-bit codecs on a row in registers.
#pragma once

#include "la_layer.hpp"

namespace la {

constexpr int kPiece = 8;

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        widen(load16(p), v);
    } else {
        float a[4], b[4];
        widen(load16(p), a);
        widen(load16(p + 4), b);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        store16(p, narrow(v));
    } else {
        store16(p, uv4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
        store16(p + 4, uv4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])});
    }
}
__device__ __forceinline__ void load_w(const void* w, int dtype, int col, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = 1.0f;
    } else if (dtype == LA_BF16) {
        load8(static_cast<const uint16_t*>(w) + col, v);
    } else {
        load8(static_cast<const float*>(w) + col, v);
    }
}

// The larger of a magnitude and |b|, a NaN above every number (fmaxf would drop it).
__device__ __forceinline__ float larger_abs(float a, float b) {
    const uint32_t u = __float_as_uint(a), v = __float_as_uint(b) & 0x7FFFFFFFu;
    return __uint_as_float(u > v ? u : v);
}

// Sum over the row's lanes, the same bits in each of them.
template <int LANES>
__device__ __forceinline__ float row_sum(float x, float* lds) {
    if constexpr (LANES <= 64) return group_sum<LANES>(x);
    x = group_sum<64>(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}
// Two sums at once, by one barrier: `lds` is another eight words in the next call.
template <int LANES>
__device__ __forceinline__ void row_sums(float& a, float& b, float* lds) {
    a = group_sum<(LANES < 64 ? LANES : 64)>(a);
    b = group_sum<(LANES < 64 ? LANES : 64)>(b);
    if constexpr (LANES <= 64) return;
    if ((threadIdx.x & 63) == 0) {
        lds[threadIdx.x >> 6] = a;
        lds[4 + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    b = (lds[4] + lds[5]) + (lds[6] + lds[7]);
}
__device__ __forceinline__ double join64(uint32_t lo, uint32_t hi) {
    return __builtin_bit_cast(double, static_cast<uint64_t>(lo) | (static_cast<uint64_t>(hi) << 32));
}
template <int CTRL>
__device__ __forceinline__ double dpp_double(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return join64(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xF, 0xF, true),
                  __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xF, 0xF, true));
}
// The sum of doubles, by the exchanges of group_sum (by shuffles: 14.2 us against 12.7 for 40000 rows of 128).
template <int LANES>
__device__ __forceinline__ double row_sum_wide(double x, double* lds) {
    if (LANES >= 2) x += dpp_double<kDppXor1>(x);
    if (LANES >= 4) x += dpp_double<kDppXor2>(x);
    if (LANES >= 8) x += dpp_double<kDppHalfMirror>(x);
    if (LANES >= 16) x += dpp_double<kDppMirror>(x);
    if (LANES >= 32) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint32_t a = static_cast<uint32_t>(u), b = static_cast<uint32_t>(u >> 32);
        const auto lo = __builtin_amdgcn_permlane16_swap(a, a, false, false), hi = __builtin_amdgcn_permlane16_swap(b, b, false, false);
        x = join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
    }
    if (LANES >= 64) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint32_t a = static_cast<uint32_t>(u), b = static_cast<uint32_t>(u >> 32);
        const auto lo = __builtin_amdgcn_permlane32_swap(a, a, false, false), hi = __builtin_amdgcn_permlane32_swap(b, b, false, false);
        x = join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
    }
    if constexpr (LANES <= 64) return x;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}
template <int LANES>
__device__ __forceinline__ float row_max(float x, float* lds) {
    if constexpr (LANES <= 64) return group_max_abs<LANES>(x);
    x = group_max_abs<64>(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0];
#pragma unroll
    for (int k = 1; k < LANES / 64; k++) x = larger_abs(x, lds[k]);
    return x;
}

// 1 / sqrt(m), correct to about an ulp: the hardware's estimate and one Newton step (skipped
// where the estimate is 0, infinite or NaN).
__device__ __forceinline__ float rsqrt_fine(float m) {
    const float r = __builtin_amdgcn_rsqf(m);
    const float e = __builtin_fmaf(-m * r, r, 1.0f);
    const float y = __builtin_fmaf(0.5f * r, e, r);
    return (m > 1e-35f && m < 1e35f) ? y : 1.0f / sqrtf(m);
}

// Where a row's codes and scales go (each may be null), and the columns that share a scale (0: the row).
struct CodeOut {
    int d, group;
    uint8_t* codes;
    float* scales;
};

// Quantizes a row in registers: h becomes the values that its codes stand for.  amax[c]: the largest
// magnitude of piece c.
template <int QDQ, int LANES, int CH>
__device__ __forceinline__ void emit_codes(const CodeOut& o, int l, int row, size_t base, float (&h)[CH][8], float (&amax)[CH], float* lds) {
    if (o.group == 0) {
        float m = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; c++) m = larger_abs(m, amax[c]);
        m = row_max<LANES>(m, lds);
#pragma unroll
        for (int c = 0; c < CH; c++) amax[c] = m;
    } else {  // a row of LANES * 8 columns or more holds whole groups; in a shorter one a group may be the row
#pragma unroll
        for (int c = 0; c < CH; c++) {
            amax[c] = group_max_abs<2>(amax[c]);
            if (o.group >= 32) amax[c] = larger_abs(amax[c], dpp<kDppXor2>(amax[c]));
            if (o.group >= 64) amax[c] = larger_abs(amax[c], dpp<kDppHalfMirror>(amax[c]));
            if (o.group >= 128) amax[c] = larger_abs(amax[c], dpp<kDppMirror>(amax[c]));
        }
    }
    const int per_row = o.group ? o.d / o.group : 1;
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int col = (c * LANES + l) * kPiece;
        if (col >= o.d) continue;
        float s, y;
        uint32_t word[2] = {0, 0};
        // a NaN in the group: its maximum, its scale and every value that its codes stand for
        const bool none = amax[c] != amax[c];
        bool fast = QDQ == LA_QDQ_INT8_GROUP ? int8_scale_recip(amax[c], s, y) : e4m3_scale_recip(amax[c], s, y);
        if (none) s = amax[c], fast = false;
        if (fast) {  // numbers, whose quotients no code's range leaves
            if constexpr (QDQ == LA_QDQ_INT8_GROUP) {
                uint32_t q[8];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float r = int8_code_fast(h[c][e], s, y);
                    q[e] = __float_as_uint(r + 12582912.0f);  // (1.5 x 2^23: the integer in the low byte)
                    h[c][e] = r * s;
                }
#pragma unroll
                for (int k = 0; k < 2; k++)
                    word[k] = __builtin_amdgcn_perm(q[4 * k + 1], q[4 * k], 0x0c0c0400u) | __builtin_amdgcn_perm(q[4 * k + 3], q[4 * k + 2], 0x04000c0cu);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float a = fminf(fmaxf(quot_rn_fast(h[c][e], s, y), -448.0f), 448.0f);
                    const float b = fminf(fmaxf(quot_rn_fast(h[c][e + 1], s, y), -448.0f), 448.0f);
                    const uint32_t k = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false)) & 0xFFFFu;
                    word[e >> 2] |= k << (8 * (e & 3));
                    h[c][e] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(k), 0) * s;
                    h[c][e + 1] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(k), 1) * s;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float x = h[c][e] / s;
                const bool number = x == x;  // (of a quotient without one: code 0, or E4M3's NaN)
                if constexpr (QDQ == LA_QDQ_INT8_GROUP) {
                    const float q = number ? fminf(fmaxf(rintf(x), -127.0f), 127.0f) : x;
                    word[e >> 2] |= (number ? static_cast<uint32_t>(static_cast<int>(q)) & 0xFFu : 0u) << (8 * (e & 3));
                    h[c][e] = q * s;
                } else {
                    const float a = number ? fminf(fmaxf(x, -448.0f), 448.0f) : x;
                    const uint32_t k = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(a, a, 0, false)) & 0xFFu;
                    word[e >> 2] |= k << (8 * (e & 3));
                    h[c][e] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(k), 0) * s;
                }
            }
        }
        if (o.codes) *reinterpret_cast<uv2*>(o.codes + base + col) = uv2{word[0], word[1]};
        if (o.scales) {
            if (o.group ? col % o.group == 0 : col == 0)
                o.scales[static_cast<size_t>(row) * per_row + (o.group ? col / o.group : 0)] = s;
        }
    }
}

}  // namespace la
