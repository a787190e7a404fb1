// Lane sums and the gate's functions of the norms around a block.
#pragma once

#include "la_norm.hpp"
#include "la_proj.hpp"

namespace la {

// Sum over aligned groups of `n` lanes (a power of two up to 64, the same for the whole launch).
__device__ __forceinline__ float sum_lanes(float x, int n) {
    if (n >= 2) x = x + dpp<kDppXor1>(x);
    if (n >= 4) x = x + dpp<kDppXor2>(x);
    if (n >= 8) x = x + dpp<kDppHalfMirror>(x);
    if (n >= 16) x = x + dpp<kDppMirror>(x);
    if (n >= 32) { Pair p = swap16(x); x = p.a + p.b; }
    if (n >= 64) { Pair p = swap32(x); x = p.a + p.b; }
    return x;
}
__device__ __forceinline__ double sum_lanes(double x, int n) {
    if (n >= 2) x += dpp_double<kDppXor1>(x);
    if (n >= 4) x += dpp_double<kDppXor2>(x);
    if (n >= 8) x += dpp_double<kDppHalfMirror>(x);
    if (n >= 16) x += dpp_double<kDppMirror>(x);
    if (n >= 32) x += __shfl_xor(x, 16);
    if (n >= 64) x += __shfl_xor(x, 32);
    return x;
}
// Sum over the row's lanes, in one barrier: `lds` belongs to this call alone.
template <int LANES, class S>
__device__ __forceinline__ S sum_row(S x, S* lds) {
    x = sum_lanes(x, LANES < 64 ? LANES : 64);
    if constexpr (LANES <= 64) return x;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    S s = lds[0];
#pragma unroll
    for (int k = 1; k < LANES / 64; k++) s += lds[k];
    return s;
}

// act(z), and its derivative.
template <class T>
__device__ __forceinline__ float gate_of(float z, int gate) {
    const float s = sigmoid_for<T>(z);
    return gate == LA_GATE_SILU ? (z < -89.0f ? 0.0f : z * s) : s;
}
template <class T>
__device__ __forceinline__ void gate_both(float z, int gate, float& g, float& slope) {
    const float s = sigmoid_for<T>(z);
    if (gate == LA_GATE_SILU) {
        g = z < -89.0f ? 0.0f : z * s;  // (s is 0 there: of z = -inf too)
        slope = z < -89.0f ? 0.0f : s * (1.0f + z * (1.0f - s));
    } else {
        g = s;
        slope = s * sigmoid_for<T>(-z);  // (1 - s keeps 24 - 1.44 z bits of what is left at large z)
    }
}

}  // namespace la
