// Internal interface of the operators between two recurrences (matrix product of 8-bit codes, norms
// around a block): the launchers behind la_proj.cpp.
#pragma once

#include "../../include/la_proj.h"
#include "la_layer.hpp"

namespace la {

struct LinearArgs {
    const int8_t* x = nullptr;
    const float* xs = nullptr;
    const int8_t* w = nullptr;
    const float* ws = nullptr;
    const void* bias = nullptr;
    void* y = nullptr;
    const void* dy = nullptr;
    void* dx = nullptr;
    void* dw = nullptr;
    float* dbias = nullptr;
    char* work = nullptr;
};
hipError_t launch_linear_fwd(const la_linear_config& c, const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_bwd(const la_linear_config& c, const LinearArgs& a, hipStream_t s);
size_t linear_bwd_workspace(const la_linear_config& c);

struct GateArgs {
    const void* x = nullptr;
    const void* z = nullptr;
    const void* w_post = nullptr;
    const void* alpha = nullptr;
    const void* res = nullptr;
    const void* w_pre = nullptr;
    void* h = nullptr;  // the backward's input
    void* y = nullptr;
    void* codes = nullptr;
    float* scales = nullptr;
    const void* dy = nullptr;
    const void* dh = nullptr;
    void* dx = nullptr;
    void* dz = nullptr;
    void* dres = nullptr;
    float* dw_post = nullptr;
    float* dalpha = nullptr;
    float* dw_pre = nullptr;
    float* part = nullptr;
};
// Lanes that hold a row of the forward: pieces of 8 columns on 8 to 64 lanes of a wave, then a workgroup of whole
// waves, with two pieces a lane and more from about 384 pieces on.
inline int gate_lanes(int d) {
    const int pieces = d / 8;
    if (pieces <= 64) return pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    return pieces <= 128 ? 128 : pieces <= 192 ? 192 : pieces <= 256 ? 256 : pieces <= 384 ? 384 : 256;
}
hipError_t launch_gate_fwd(const la_gate_norm_config& c, const GateArgs& a, hipStream_t s);
hipError_t launch_gate_bwd(const la_gate_norm_config& c, const GateArgs& a, hipStream_t s);
size_t gate_bwd_workspace(const la_gate_norm_config& c);

}  // namespace la
