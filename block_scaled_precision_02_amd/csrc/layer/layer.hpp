// layer.hpp -- launchers of the decoder-layer operators.  Arguments are
// checked by the C entry points (layer_api.cpp) before these are called.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace qgemm {

// RMS norm with 8-bit (or e2m1) output.
enum NormOut { NORM_I8_ROW = 0, NORM_F8_ROW = 1, NORM_F8_BLOCK = 2, NORM_MX_E4M3 = 3, NORM_MX_E2M1 = 4 };
struct NormArgs {
    const uint16_t *X, *R, *gamma;   // bf16; R NULL: no residual
    uint16_t *Rout;                  // bf16(X + R), NULL: not written
    uint8_t *Q;
    void *S;                         // fp32 [M], fp32 [M, K/128] or ue8m0 [M, K/32]
    int64_t ldx, ldr, ldo, ldq, lds; // elements; ldq, MX lds bytes
    int M, K;
    float eps;
};
hipError_t launch_rmsnorm_quant(int out, const NormArgs &a, hipStream_t s);

}  // namespace qgemm
