// experts.hpp -- launchers of the operators of a layer of experts.  Arguments
// are checked by the C entry points (experts_api.cpp) before these are called.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace qgemm {

constexpr int MOE_MAX_EXPERTS = 1024;
constexpr int MOE_MAX_K = 64;

// Choices in order of experts.
struct SortArgs {
    const int32_t *ids;                       // [slots]
    int32_t *offsets, *order, *position;      // [experts + 1], [slots], [slots]
    int32_t *hist;                            // workspace: [blocks, experts], one workgroup's counts a row
    int slots, experts;
    int blocks, chunk;                        // the plan (sort_plan): workgroups, slots of each
};
// Fills the plan; returns the workspace bytes it needs.
int64_t sort_plan(SortArgs &a);
hipError_t launch_moe_sort(const SortArgs &a, hipStream_t s);

// Rows to the experts and back.
struct ExchangeArgs {
    const uint16_t *X;                        // [tokens, H]: gather: x; combine: residual or NULL; gradient: dout
    const uint16_t *Y;                        // [rows, H]: combine and gradient: the experts' rows
    uint16_t *O;                              // gather, gradient: [rows, H]; combine: [tokens, H]
    const float *W;                           // [tokens, k] or NULL: ones
    float *dW;                                // [tokens, k]
    const int32_t *position;                  // [tokens, k]
    int64_t ldx, ldy, ldo;
    int64_t rows;
    int tokens, k, H;
};
hipError_t launch_moe_gather(const ExchangeArgs &a, hipStream_t s);
hipError_t launch_moe_combine(const ExchangeArgs &a, hipStream_t s);
hipError_t launch_moe_combine_grad(const ExchangeArgs &a, hipStream_t s);

// silu(gate) * up with output in 8 bits (out: NormOut).
struct SwigluArgs {
    const uint16_t *X;                        // [M, 2 I]: gate, up
    uint8_t *Q;
    void *S;
    const int32_t *count;                     // rows to do, on the device; NULL: M
    int64_t ldx, ldq, lds;
    int64_t row0;                             // the launch's first row
    int M, I;
    unsigned row_mul, row_shift;              // the launch's: n / (I / 8) = n * row_mul >> 32 + row_shift
};
hipError_t launch_swiglu_quant(int out, const SwigluArgs &a, hipStream_t s);

// One scaled product per expert over its rows.
struct GroupedArgs {
    const uint8_t *A, *B;                     // [rows of A, K] and [experts, N, K], codes
    const void *SA, *SB;                      // the path's scales
    const uint16_t *bias;                     // [experts, N] or NULL
    uint16_t *C;                              // [rows, N]
    const int32_t *offsets, *order;           // [experts + 1]; [rows] or NULL
    int64_t lda, ldb, ldc, b_expert;          // bytes, bytes, elements, bytes
    int64_t a_rows, rows;
    int top_k, experts, N, K;
};
// path: qgemm::Path (I8, F8, MX8, MX4, F8B)
int grouped_tile_id(int path, const GroupedArgs &a); // by rows, experts and N
bool grouped_fits(int path, const GroupedArgs &a);   // in one launch
hipError_t launch_grouped(int path, const GroupedArgs &a, hipStream_t s);

}  // namespace qgemm
