// Internal interface of the layer operators (convolution, selective scan, norm): the launchers
// behind la_layer.cpp and the device helpers that they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/la_layer.h"
#include "la_device.hpp"

namespace la {

// la_api.cpp: sets the calling thread's la_last_error and returns s.
la_status report(la_status s, const char* detail);

struct ConvArgs {
    const int32_t* cu = nullptr;  // null: dense [B][T]
    const void* x = nullptr;
    const void* w = nullptr;
    const void* bias = nullptr;
    const void* s0 = nullptr;
    void* y = nullptr;
    void* sT = nullptr;
    const void* dy = nullptr;
    const void* dsT = nullptr;
    void* dx = nullptr;
    float* dw = nullptr;
    float* dbias = nullptr;
    void* ds0 = nullptr;
    float* part = nullptr;
    // decode step
    void* state = nullptr;
    const int32_t* slots = nullptr;
    int n_slots = 0;
};
hipError_t launch_conv_fwd(const la_conv_config& c, const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_bwd(const la_conv_config& c, const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(const la_conv_config& c, const ConvArgs& a, hipStream_t s);
size_t conv_bwd_workspace(const la_conv_config& c);

struct NormArgs {
    const void* x = nullptr;
    const void* res = nullptr;
    const void* w = nullptr;
    void* res_out = nullptr;
    void* y = nullptr;
    void* codes = nullptr;
    float* scales = nullptr;
    const void* dy = nullptr;
    const void* dres = nullptr;
    void* dx = nullptr;
    float* dw = nullptr;
    float* part = nullptr;
};
hipError_t launch_norm_fwd(const la_norm_config& c, const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const la_norm_config& c, const NormArgs& a, hipStream_t s);
size_t norm_bwd_workspace(const la_norm_config& c);

struct ScanArgs {
    const int32_t* cu = nullptr;
    const void* x = nullptr;
    const void* dt = nullptr;
    const float* A = nullptr;
    const void* b = nullptr;
    const void* c = nullptr;
    const float* D = nullptr;
    const float* bias = nullptr;
    const float* S0 = nullptr;
    void* y = nullptr;
    float* ST = nullptr;
    const void* dy = nullptr;
    const float* dST = nullptr;
    void* dx = nullptr;
    void* ddt = nullptr;
    float* dA = nullptr;
    void* db = nullptr;
    void* dc = nullptr;
    float* dD = nullptr;
    float* dbias = nullptr;
    float* dS0 = nullptr;
    char* ws = nullptr;
    // decode step
    float* S = nullptr;
    const int32_t* slots = nullptr;
    int n_slots = 0;
};
hipError_t launch_scan_fwd(const la_scan_config& c, const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd(const la_scan_config& c, const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_step(const la_scan_config& c, const ScanArgs& a, hipStream_t s);
size_t scan_fwd_workspace(const la_scan_config& c);
size_t scan_bwd_workspace(const la_scan_config& c, bool packed);
int64_t scan_bwd_slots(const la_scan_config& c, bool packed);  // chunks of 64 tokens in its workspace
// Workgroups of a launch of 512 threads, and half of those of one of 256: a grid has below 2^32 threads.
constexpr int64_t kMaxUnits = static_cast<int64_t>(1) << 23;

// out[i] = sum in double over p < parts of part[p cols + i], p in order within each of 32 interleaved
// partial sums (a fixed order: the result does not depend on scheduling).  Columns from
// `split` on go to out2 (may be null).
hipError_t launch_reduce_parts(const float* part, int parts, int cols, float* out, int split, float* out2,
                               hipStream_t s);

// Zeros to `width` elements of each of `rows` rows `ld` elements apart (out null: nothing).
hipError_t launch_zero_rows(void* out, int dtype, int64_t rows, int64_t width, int64_t ld, hipStream_t s);

// ------------------------------------------------------------------ device helpers
typedef float fv4 __attribute__((ext_vector_type(4)));
typedef uint32_t uv4 __attribute__((ext_vector_type(4)));
typedef uint32_t uv2 __attribute__((ext_vector_type(2)));

// The storage types: bf16 bits or float.  kVec elements are one 16-byte access.
template <class T>
struct Io;
template <>
struct Io<uint16_t> {
    static constexpr int kVec = 8;
    static constexpr int kCode = LA_BF16;
};
template <>
struct Io<float> {
    static constexpr int kVec = 4;
    static constexpr int kCode = LA_F32;
};

// Two bf16 halves of a word, widened.
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
typedef float fv2 __attribute__((ext_vector_type(2)));
typedef __bf16 bv2 __attribute__((ext_vector_type(2)));
// Two floats rounded to bf16 (nearest, ties to even) in one word.
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(fv2{a, b}, bv2));
}

// 16 bytes of a row, widened / rounded.
__device__ __forceinline__ void widen(uv4 r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = lo16(r[i]);
        v[2 * i + 1] = hi16(r[i]);
    }
}
__device__ __forceinline__ void widen(uv4 r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ uv4 narrow(const float (&v)[8]) {
    return uv4{pack16(v[0], v[1]), pack16(v[2], v[3]), pack16(v[4], v[5]), pack16(v[6], v[7])};
}
__device__ __forceinline__ uv4 narrow(const float (&v)[4]) {
    return uv4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}
template <class T>
__device__ __forceinline__ uv4 load16(const T* p) {
    return *reinterpret_cast<const uv4*>(p);
}
template <class T>
__device__ __forceinline__ void store16(T* p, uv4 v) {
    *reinterpret_cast<uv4*>(p) = v;
}

// exp(x) within about 2 ulp for x in [-87, 88]: the product with log2(e) in two parts, the
// second applied to first order.
__device__ __forceinline__ float exp_fine(float x) {
    constexpr float kL2E = 1.44269502162933349609375f, kL2Elo = 1.925963033500011e-08f, kLn2 = 0.693147180559945309f;
    const float t = x * kL2E;
    const float e = __builtin_fmaf(x, kL2Elo, __builtin_fmaf(x, kL2E, -t));
    const float r = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(r, e * kLn2, r);
}

// 1 / (1 + exp(-x)) within (|x| + 2) 2^-23 of itself: the hardware's exponential of the rounded
// product and its reciprocal, no correction of either (the bf16 convolution is bound by its
// instructions where memory keeps up, and rounds the result to 2^-8).  0 from x = -89 down, where
// the exponential is infinite.
__device__ __forceinline__ float sigmoid_fine(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504088896341f));
}
// The same within 4 2^-23 of itself, for results kept in FP32: the product with log2(e) in two parts
// as in exp_fine and one Newton step for the reciprocal, each skipped where it would meet an infinity.
__device__ __forceinline__ float sigmoid_full(float x) {
    constexpr float kL2E = 1.44269502162933349609375f, kL2Elo = 1.925963033500011e-08f, kLn2 = 0.693147180559945309f;
    const float t = x * -kL2E;
    const float lo = __builtin_fmaf(x, -kL2Elo, __builtin_fmaf(x, -kL2E, -t));
    const float r = __builtin_amdgcn_exp2f(t);
    const float d = 1.0f + (fabsf(t) < 126.0f ? __builtin_fmaf(r, lo * kLn2, r) : r);
    const float q = __builtin_amdgcn_rcpf(d);
    return d < 0x1p126f ? __builtin_fmaf(__builtin_fmaf(-d, q, 1.0f), q, q) : q;
}
// By the type that holds the result.
template <class T>
__device__ __forceinline__ float sigmoid_for(float x) {
    if constexpr (sizeof(T) == 4) return sigmoid_full(x);
    else return sigmoid_fine(x);
}

// Sequence b of a packing, clamped to [0, T].
struct Span {
    int begin, end;
};
__device__ __forceinline__ Span packed_span(const int32_t* cu, int b, int T) {
    int lo = cu[b], hi = cu[b + 1];
    lo = lo < 0 ? 0 : (lo > T ? T : lo);
    hi = hi < lo ? lo : (hi > T ? T : hi);
    return {lo, hi};
}
// The last b with cu[b] <= t, or 0: the sequence of token t if t lies in one.  Eight boundaries a
// step, read together: two reads' latency for 64 sequences, four for 4096.
__device__ __forceinline__ int packed_find(const int32_t* cu, int B, int t) {
    int lo = 0, n = B;  // among lo .. lo + n - 1, cu[lo] <= t or lo = 0
    while (n > 1) {
        const int step = (n + 7) / 8;
        int at[7], k = 0;
#pragma unroll
        for (int i = 0; i < 7; i++) at[i] = cu[lo + (step * (i + 1) < n ? step * (i + 1) : 0)];
#pragma unroll
        for (int i = 0; i < 7; i++) k = step * (i + 1) < n && at[i] <= t ? i + 1 : k;
        lo += k * step;
        n = n - k * step < step ? n - k * step : step;
    }
    return lo;
}

}  // namespace la
