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

// The paged 8-bit cache (kv8_dev.hpp has the layout).
enum Kv8Fmt { KV8_E4M3 = 0, KV8_I8 = 1 };
struct Kv8Append {
    uint8_t *ck, *cv;
    float *sk, *sv;                   // [blocks, kv_heads]
    const uint16_t *K, *V;            // bf16 [tokens, kv_heads, dim], token strides ldk, ldv elements
    const int32_t *table, *cu, *lens; // [batch, ldt], [batch + 1], [batch]
    int64_t ldk, ldv, ldt, tokens;
    int blocks, kv_heads, dim, bs, fmt, width, batch, max_q;
    int at;                           // the launch's first block of a sequence's new tokens
};
hipError_t launch_kv8_append(const Kv8Append &a, hipStream_t s);

struct Kv8Attn {
    const uint8_t *ck, *cv;
    const float *sk, *sv;
    const uint16_t *Q;                // bf16 [tokens, heads, dim], token stride ldq elements
    uint16_t *O;                      // the same, ldo
    const int32_t *table, *cu, *lens;
    float *part, *stat;               // workspace of a split call
    int64_t ldq, ldo, ldt, tokens;
    float scale2;                     // softmax scale times log2(e)
    int blocks, kv_heads, group, dim, bs, fmt, width, batch, max_q, max_kv, causal, window;
    // the plan (kv8_plan)
    int kernel;                       // 0 streaming (few rows), 1 tiled (many rows)
    int nt;                           // streaming: 16-row tiles a wave
    int waves;                        // waves a workgroup (tiled: of 32 rows each)
    int row_tiles;                    // of the longest sequence, per kv head
    int split_steps, splits;          // steps of 64 tokens a split, splits
};
// Fills the plan; returns the workspace bytes it needs.
int64_t kv8_plan(Kv8Attn &a);
hipError_t launch_kv8_attention(const Kv8Attn &a, hipStream_t s);
hipError_t launch_kv8_tile(const Kv8Attn &a, hipStream_t s);   // the tiled kernel alone
// Waves a SIMD that it is built for, by head_dim / 64 and waves a workgroup; 0:
// not built.
int kv8_tile_occupancy(int dc, int waves);

// bf16 rows times 4-bit weights (M <= 64).
struct W4Args {
    const uint16_t *X;                // bf16 [M, K], row stride ldx elements
    const uint8_t *W;                 // [N, K/2] bytes, row stride ldw
    const void *S;                    // bf16 [N, K/group], or ue8m0 [N / srows, K/32]
    const uint8_t *Z;                 // [N, K/group] or NULL
    const uint16_t *bias;             // bf16 [N] or NULL
    uint16_t *Y;                      // bf16 [M, N], row stride ldy elements
    int64_t ldx, ldw, ldy;
    int M, N, K, group, srows;        // group 0: MX
};
hipError_t launch_w4_matvec(const W4Args &a, hipStream_t s);

}  // namespace qgemm
