// layer_api.cpp -- C entry points of the decoder-layer operators: argument
// checks, then the launchers of layer.hpp.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../qgemm_host.hpp"
#include "layer.hpp"

using namespace qgemm;

namespace {

qgemm_status check_rows(const char *name, const void *p, int64_t ld, int64_t K)
{
    if (!p)
        return fail(QGEMM_ERR_NULL_POINTER, "%s is NULL", name);
    if (!aligned(p, 16))
        return fail(QGEMM_ERR_BAD_LAYOUT, "%s is not 16-byte aligned", name);
    if (ld < K || ld % 8 || ld >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_LAYOUT, "row stride of %s, %lld elements: need >= %lld, a multiple of 8, below 2^31",
                    name, (long long)ld, (long long)K);
    return QGEMM_OK;
}

// The shape of a norm with quantised output.
qgemm_status check_norm_shape(int out, float eps, int64_t M, int64_t K)
{
    if (M < 0 || K <= 0)
        return fail(QGEMM_ERR_BAD_SHAPE, "M=%lld K=%lld: need M>=0, K>0", (long long)M, (long long)K);
    const int64_t unit = out == NORM_F8_BLOCK ? 128 : 32;
    if (K % unit)
        return fail(QGEMM_ERR_BAD_SHAPE, "K=%lld is not a multiple of %lld", (long long)K, (long long)unit);
    if (M >= LD_LIMIT || K >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_SHAPE, "M and K must stay below 2^31");
    if (!(eps >= 0.0f))
        return fail(QGEMM_ERR_BAD_SHAPE, "eps=%g: need a number >= 0", (double)eps);
    return QGEMM_OK;
}

// Its codes and scales.
qgemm_status check_norm_out(int out, const void *Q, int64_t ldq, const void *S, int64_t lds, int64_t s_row, int64_t K)
{
    if (!Q)
        return fail(QGEMM_ERR_NULL_POINTER, "Q is NULL");
    const int64_t q_row = out == NORM_MX_E2M1 ? K / 2 : K;
    if (!aligned(Q, 16) || ldq < q_row || ldq % 16 || ldq >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_LAYOUT,
                    "Q must be 16-byte aligned with ldq=%lld bytes >= %lld, a multiple of 16, below 2^31",
                    (long long)ldq, (long long)q_row);
    if (!S)
        return fail(QGEMM_ERR_NULL_POINTER, "the scale array is NULL");
    if (out <= NORM_F8_BLOCK && !aligned(S, 4))
        return fail(QGEMM_ERR_BAD_LAYOUT, "the scale array is not 4-byte aligned");
    if (out >= NORM_F8_BLOCK && (lds < s_row || lds >= LD_LIMIT))
        return fail(QGEMM_ERR_BAD_LAYOUT, "lds=%lld: need >= %lld, below 2^31", (long long)lds, (long long)s_row);
    return QGEMM_OK;
}

// out: NormOut; the scale array's alignment and row length are the caller's.
qgemm_status norm_common(int out, const uint16_t *X, int64_t ldx, const uint16_t *R, int64_t ldr,
                         const uint16_t *gamma, float eps, uint16_t *Rout, int64_t ldo, void *Q, int64_t ldq, void *S,
                         int64_t lds, int64_t s_row, int64_t M, int64_t K, void *stream)
{
    TRY(check_norm_shape(out, eps, M, K));
    if (M == 0)
        return QGEMM_OK;
    TRY(check_rows("X", X, ldx, K));
    if (R)
        TRY(check_rows("R", R, ldr, K));
    if (Rout)
        TRY(check_rows("Rout", Rout, ldo, K));
    TRY(check_rows("gamma", gamma, K, K));
    TRY(check_norm_out(out, Q, ldq, S, lds, s_row, K));
    TRY(check_device());
    const NormArgs a = {X, R, gamma, Rout, (uint8_t *)Q, S, ldx, ldr, ldo, ldq, lds, (int)M, (int)K, eps};
    return launch([&] { return launch_rmsnorm_quant(out, a, (hipStream_t)stream); });
}

qgemm_status postnorm_common(int out, const qgemm_postnorm *n, void *Q, int64_t ldq, void *S, int64_t lds,
                             int64_t s_row, int64_t M, int64_t K, void *stream)
{
    if (!n)
        return fail(QGEMM_ERR_NULL_POINTER, "the norm's arguments are NULL");
    TRY(check_norm_shape(out, n->eps, M, K));
    if (!std::isfinite(n->alpha))
        return fail(QGEMM_ERR_BAD_SHAPE, "alpha is not finite");
    if (M == 0)
        return QGEMM_OK;
    TRY(check_rows("Y", n->Y, n->ldy, K));
    TRY(check_rows("R", n->R, n->ldr, K));
    if (n->Rout)
        TRY(check_rows("Rout", n->Rout, n->ldo, K));
    TRY(check_rows("gamma_post", n->gamma_post, K, K));
    if (n->gate)
        TRY(check_rows("gate", n->gate, K, K));
    TRY(check_rows("gamma", n->gamma, K, K));
    TRY(check_norm_out(out, Q, ldq, S, lds, s_row, K));
    TRY(check_device());
    const PostnormArgs a = {n->Y, n->R, n->gamma_post, n->gate, n->gamma, n->Rout, (uint8_t *)Q, S, n->ldy, n->ldr,
                            n->ldo, ldq, lds, (int)M, (int)K, n->eps, n->alpha};
    return launch([&] { return launch_postnorm_quant(out, a, (hipStream_t)stream); });
}

// ------------------------------------------------------------ 8-bit cache

qgemm_status check_cache(const qgemm_kv8_cache *c)
{
    if (!c)
        return fail(QGEMM_ERR_NULL_POINTER, "cache is NULL");
    if (c->fmt != QGEMM_KV8_E4M3 && c->fmt != QGEMM_KV8_I8)
        return fail(QGEMM_ERR_BAD_FORMAT, "unknown cache format %d", c->fmt);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 192 && c->head_dim != 256)
        return fail(QGEMM_ERR_BAD_SHAPE, "head_dim=%d: need 64, 128, 192 or 256", c->head_dim);
    if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
        return fail(QGEMM_ERR_BAD_SHAPE, "block=%d tokens: need 16, 32, 64 or 128", c->block);
    if (c->kv_heads <= 0 || c->kv_heads > 32767)
        return fail(QGEMM_ERR_BAD_SHAPE, "kv_heads=%d: need 1 to 32767", c->kv_heads);
    if (c->num_blocks <= 0 || c->num_blocks >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_SHAPE, "num_blocks=%lld: need 1 to 2^31 - 1", (long long)c->num_blocks);
    if (!c->k || !c->v || !c->k_scale || !c->v_scale)
        return fail(QGEMM_ERR_NULL_POINTER, "a cache array is NULL");
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return fail(QGEMM_ERR_BAD_LAYOUT, "cache codes must be 16-byte aligned, scales 4-byte");
    return QGEMM_OK;
}

// Sequences: block table, new-token offsets, lengths.
qgemm_status check_seqs(const int32_t *table, int64_t ldt, int64_t width, const int32_t *cu, const int32_t *lens,
                        int64_t tokens, int64_t batch, int64_t max_q)
{
    if (batch < 0 || batch > 65535)
        return fail(QGEMM_ERR_BAD_SHAPE, "batch=%lld: need 0 to 65535", (long long)batch);
    if (tokens < 0 || tokens >= LD_LIMIT || max_q < 0 || max_q > tokens)
        return fail(QGEMM_ERR_BAD_SHAPE, "tokens=%lld max_q=%lld: need 0 <= max_q <= tokens < 2^31", (long long)tokens,
                    (long long)max_q);
    if (width < 0 || width >= LD_LIMIT || ldt < width)
        return fail(QGEMM_ERR_BAD_SHAPE, "block table rows of %lld entries, stride %lld: need 0 <= entries <= stride",
                    (long long)width, (long long)ldt);
    if (batch == 0 || max_q == 0)
        return QGEMM_OK;
    if (!table || !cu || !lens)
        return fail(QGEMM_ERR_NULL_POINTER, "block_table, cu_seqlens or kv_lens is NULL");
    if (!aligned(table, 4) || !aligned(cu, 4) || !aligned(lens, 4))
        return fail(QGEMM_ERR_BAD_LAYOUT, "block_table, cu_seqlens and kv_lens must be 4-byte aligned");
    return QGEMM_OK;
}

qgemm_status check_attn_shape(const qgemm_kv8_cache *c, int64_t heads, int64_t max_kv, int causal, int64_t window)
{
    if (heads <= 0 || heads % c->kv_heads || heads > 65535)
        return fail(QGEMM_ERR_BAD_SHAPE, "heads=%lld: need a multiple of kv_heads=%d, at most 65535", (long long)heads,
                    c->kv_heads);
    if (max_kv < 0 || max_kv >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_SHAPE, "max_kv=%lld: need 0 to 2^31 - 1", (long long)max_kv);
    if (window < 0 || window >= LD_LIMIT || (window > 0 && !causal))
        return fail(QGEMM_ERR_BAD_SHAPE, "window=%lld: need 0 (none) or a length, with causal", (long long)window);
    return QGEMM_OK;
}

Kv8Attn attn_args(const qgemm_kv8_cache *c, int64_t tokens, int64_t batch, int64_t heads, int64_t max_q,
                  int64_t max_kv, int causal, int64_t window)
{
    Kv8Attn a = {};
    a.ck = (const uint8_t *)c->k;
    a.cv = (const uint8_t *)c->v;
    a.sk = c->k_scale;
    a.sv = c->v_scale;
    a.tokens = tokens;
    a.blocks = (int)c->num_blocks;
    a.kv_heads = c->kv_heads;
    a.group = (int)(heads / c->kv_heads);
    a.dim = c->head_dim;
    a.bs = c->block;
    a.fmt = c->fmt;
    a.batch = (int)batch;
    a.max_q = (int)max_q;
    a.max_kv = (int)max_kv;
    a.causal = causal != 0;
    a.window = (int)window;
    return a;
}

// ------------------------------------------------------------ 4-bit matvec

constexpr int64_t W4_MAX_M = 64;

qgemm_status w4_common(W4Args a, int64_t M, int64_t N, int64_t K, int64_t group, void *stream)
{
    if (M < 0 || N < 0 || K <= 0 || M > W4_MAX_M || N >= LD_LIMIT || K >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_SHAPE, "M=%lld N=%lld K=%lld: need 0 <= M <= %lld, 0 <= N < 2^31, 0 < K < 2^31",
                    (long long)M, (long long)N, (long long)K, (long long)W4_MAX_M);
    if (group != 32 && group != 64 && group != 128)
        return fail(QGEMM_ERR_BAD_SHAPE, "group=%lld: need 32, 64 or 128", (long long)group);
    if (K % group)
        return fail(QGEMM_ERR_BAD_SHAPE, "K=%lld is not a multiple of %lld", (long long)K, (long long)group);
    if (M == 0 || N == 0)
        return QGEMM_OK;
    TRY(check_rows("X", a.X, a.ldx, K));
    if (!a.W || !a.S || !a.Y)
        return fail(QGEMM_ERR_NULL_POINTER, "%s is NULL", !a.W ? "W" : !a.S ? "the scale array" : "Y");
    if (!aligned(a.W, 16) || a.ldw < K / 2 || a.ldw % 16 || a.ldw >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_LAYOUT,
                    "W must be 16-byte aligned with ldw=%lld bytes >= %lld, a multiple of 16, below 2^31",
                    (long long)a.ldw, (long long)(K / 2));
    if (a.group && !aligned(a.S, 2))
        return fail(QGEMM_ERR_BAD_LAYOUT, "the scale array is not 2-byte aligned");
    if (!aligned(a.bias, 2) || !aligned(a.Y, 2))
        return fail(QGEMM_ERR_BAD_LAYOUT, "bias and Y must be 2-byte aligned");
    if (a.ldy < N || a.ldy >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_LAYOUT, "ldy=%lld: need >= N=%lld, below 2^31", (long long)a.ldy, (long long)N);
    TRY(check_device());
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    return launch([&] { return launch_w4_matvec(a, (hipStream_t)stream); });
}

}  // namespace

extern "C" {

qgemm_status qgemm_rmsnorm_quant_i8_rowwise(const uint16_t *X, int64_t ldx, const uint16_t *R, int64_t ldr,
                                            const uint16_t *gamma, float eps, uint16_t *Rout, int64_t ldo, int8_t *Q,
                                            int64_t ldq, float *scale, int64_t M, int64_t K, void *stream)
{
    return norm_common(NORM_I8_ROW, X, ldx, R, ldr, gamma, eps, Rout, ldo, Q, ldq, scale, 0, 0, M, K, stream);
}

qgemm_status qgemm_rmsnorm_quant_f8_pertoken(const uint16_t *X, int64_t ldx, const uint16_t *R, int64_t ldr,
                                             const uint16_t *gamma, float eps, uint16_t *Rout, int64_t ldo, uint8_t *Q,
                                             int64_t ldq, float *scale, int64_t M, int64_t K, void *stream)
{
    return norm_common(NORM_F8_ROW, X, ldx, R, ldr, gamma, eps, Rout, ldo, Q, ldq, scale, 0, 0, M, K, stream);
}

qgemm_status qgemm_rmsnorm_quant_f8_block(const uint16_t *X, int64_t ldx, const uint16_t *R, int64_t ldr,
                                          const uint16_t *gamma, float eps, uint16_t *Rout, int64_t ldo, uint8_t *Q,
                                          int64_t ldq, float *S, int64_t lds, int64_t M, int64_t K, void *stream)
{
    return norm_common(NORM_F8_BLOCK, X, ldx, R, ldr, gamma, eps, Rout, ldo, Q, ldq, S, lds, K / 128, M, K, stream);
}

qgemm_status qgemm_rmsnorm_quant_mx(qgemm_mx_fmt fmt, const uint16_t *X, int64_t ldx, const uint16_t *R, int64_t ldr,
                                    const uint16_t *gamma, float eps, uint16_t *Rout, int64_t ldo, void *Q,
                                    int64_t ldq, uint8_t *S, int64_t lds, int64_t M, int64_t K, void *stream)
{
    if (fmt != QGEMM_MX_E4M3 && fmt != QGEMM_MX_E2M1)
        return fail(QGEMM_ERR_BAD_FORMAT, "unknown MX element format %d", (int)fmt);
    return norm_common(fmt == QGEMM_MX_E4M3 ? NORM_MX_E4M3 : NORM_MX_E2M1, X, ldx, R, ldr, gamma, eps, Rout, ldo, Q,
                       ldq, S, lds, K / 32, M, K, stream);
}

qgemm_status qgemm_postnorm_quant_i8_rowwise(const qgemm_postnorm *norm, int8_t *Q, int64_t ldq, float *scale,
                                             int64_t M, int64_t K, void *stream)
{
    return postnorm_common(NORM_I8_ROW, norm, Q, ldq, scale, 0, 0, M, K, stream);
}

qgemm_status qgemm_postnorm_quant_f8_pertoken(const qgemm_postnorm *norm, uint8_t *Q, int64_t ldq, float *scale,
                                              int64_t M, int64_t K, void *stream)
{
    return postnorm_common(NORM_F8_ROW, norm, Q, ldq, scale, 0, 0, M, K, stream);
}

qgemm_status qgemm_postnorm_quant_f8_block(const qgemm_postnorm *norm, uint8_t *Q, int64_t ldq, float *S, int64_t lds,
                                           int64_t M, int64_t K, void *stream)
{
    return postnorm_common(NORM_F8_BLOCK, norm, Q, ldq, S, lds, K / 128, M, K, stream);
}

qgemm_status qgemm_postnorm_quant_mx(qgemm_mx_fmt fmt, const qgemm_postnorm *norm, void *Q, int64_t ldq, uint8_t *S,
                                     int64_t lds, int64_t M, int64_t K, void *stream)
{
    if (fmt != QGEMM_MX_E4M3 && fmt != QGEMM_MX_E2M1)
        return fail(QGEMM_ERR_BAD_FORMAT, "unknown MX element format %d", (int)fmt);
    return postnorm_common(fmt == QGEMM_MX_E4M3 ? NORM_MX_E4M3 : NORM_MX_E2M1, norm, Q, ldq, S, lds, K / 32, M, K,
                           stream);
}

qgemm_status qgemm_kv8_append(const qgemm_kv8_cache *cache, const uint16_t *K, int64_t ldk, const uint16_t *V,
                              int64_t ldv, const int32_t *block_table, int64_t ldt, int64_t width,
                              const int32_t *cu_seqlens, const int32_t *kv_lens, int64_t tokens, int64_t batch,
                              int64_t max_q, void *stream)
{
    TRY(check_cache(cache));
    TRY(check_seqs(block_table, ldt, width, cu_seqlens, kv_lens, tokens, batch, max_q));
    if (batch == 0 || max_q == 0)
        return QGEMM_OK;
    const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
    TRY(check_rows("K", K, ldk, row));
    TRY(check_rows("V", V, ldv, row));
    TRY(check_device());
    const Kv8Append a = {(uint8_t *)cache->k, (uint8_t *)cache->v, cache->k_scale, cache->v_scale, K, V, block_table,
                         cu_seqlens, kv_lens, ldk, ldv, ldt, tokens, (int)cache->num_blocks, cache->kv_heads,
                         cache->head_dim, cache->block, cache->fmt, (int)width, (int)batch, (int)max_q, 0};
    return launch([&] { return launch_kv8_append(a, (hipStream_t)stream); });
}

int64_t qgemm_kv8_attention_workspace(const qgemm_kv8_cache *cache, int64_t tokens, int64_t batch, int64_t heads,
                                      int64_t max_q, int64_t max_kv, int causal, int64_t window)
{
    if (check_cache(cache) != QGEMM_OK || check_attn_shape(cache, heads, max_kv, causal, window) != QGEMM_OK ||
        check_seqs(nullptr, 0, 0, nullptr, nullptr, tokens, 0, max_q) != QGEMM_OK || batch < 0 || batch > 65535)
        return -1;
    if (batch == 0 || max_q == 0)
        return 0;
    Kv8Attn a = attn_args(cache, tokens, batch, heads, max_q, max_kv, causal, window);
    return kv8_plan(a);
}

qgemm_status qgemm_kv8_attention(const qgemm_kv8_cache *cache, const uint16_t *Q, int64_t ldq,
                                 const int32_t *block_table, int64_t ldt, int64_t width, const int32_t *cu_seqlens,
                                 const int32_t *kv_lens, int64_t tokens, int64_t batch, int64_t heads, int64_t max_q,
                                 int64_t max_kv, float sm_scale, int causal, int64_t window, uint16_t *O, int64_t ldo,
                                 void *workspace, int64_t workspace_bytes, void *stream)
{
    TRY(check_cache(cache));
    TRY(check_seqs(block_table, ldt, width, cu_seqlens, kv_lens, tokens, batch, max_q));
    TRY(check_attn_shape(cache, heads, max_kv, causal, window));
    if (!std::isfinite(sm_scale))
        return fail(QGEMM_ERR_BAD_SHAPE, "sm_scale is not finite");
    if (batch == 0 || max_q == 0)
        return QGEMM_OK;
    TRY(check_rows("Q", Q, ldq, heads * cache->head_dim));
    TRY(check_rows("O", O, ldo, heads * cache->head_dim));
    Kv8Attn a = attn_args(cache, tokens, batch, heads, max_q, max_kv, causal, window);
    const int64_t need = kv8_plan(a);
    if (need > 0) {
        if (!workspace)
            return fail(QGEMM_ERR_NULL_POINTER, "workspace is NULL; this call needs %lld bytes", (long long)need);
        if (!aligned(workspace, 16) || workspace_bytes < need)
            return fail(QGEMM_ERR_BAD_LAYOUT, "workspace of %lld bytes: need %lld, 16-byte aligned",
                        (long long)workspace_bytes, (long long)need);
    }
    if ((int64_t)a.row_tiles * a.splits >= 65536 || max_q * 256 >= (LD_LIMIT << 1))
        return fail(QGEMM_ERR_BAD_SHAPE, "max_q=%lld with %lld heads is too large for one call", (long long)max_q,
                    (long long)heads);
    TRY(check_device());
    a.Q = Q;
    a.O = O;
    a.table = block_table;
    a.cu = cu_seqlens;
    a.lens = kv_lens;
    a.ldq = ldq;
    a.ldo = ldo;
    a.ldt = ldt;
    a.width = (int)width;
    a.scale2 = sm_scale * 1.44269504088896340736f;   // log2(e): the softmax runs on powers of two
    a.part = (float *)workspace;
    a.stat = a.part + (need > 0 ? tokens * heads * a.splits * a.dim : 0);
    return launch([&] { return launch_kv8_attention(a, (hipStream_t)stream); });
}

qgemm_status qgemm_w4_matvec_i4(const uint16_t *X, int64_t ldx, const uint8_t *W, int64_t ldw, const uint16_t *scales,
                                const uint8_t *zeros, int64_t group, const uint16_t *bias, uint16_t *Y, int64_t ldy,
                                int64_t M, int64_t N, int64_t K, void *stream)
{
    W4Args a = {};
    a.X = X;
    a.W = W;
    a.S = scales;
    a.Z = zeros;
    a.bias = bias;
    a.Y = Y;
    a.ldx = ldx;
    a.ldw = ldw;
    a.ldy = ldy;
    a.group = (int)group;
    a.srows = 1;
    return w4_common(a, M, N, K, group, stream);
}

qgemm_status qgemm_w4_matvec_mx(const uint16_t *X, int64_t ldx, const uint8_t *W, int64_t ldw, const uint8_t *scale_b,
                                qgemm_mx_bscale b_layout, const uint16_t *bias, uint16_t *Y, int64_t ldy, int64_t M,
                                int64_t N, int64_t K, void *stream)
{
    if (b_layout != QGEMM_MX_BSCALE_1x32 && b_layout != QGEMM_MX_BSCALE_32x32)
        return fail(QGEMM_ERR_BAD_FORMAT, "unknown B-scale layout %d", (int)b_layout);
    W4Args a = {};
    a.X = X;
    a.W = W;
    a.S = scale_b;
    a.bias = bias;
    a.Y = Y;
    a.ldx = ldx;
    a.ldw = ldw;
    a.ldy = ldy;
    a.group = 0;
    a.srows = (int)b_layout;
    return w4_common(a, M, N, K, 32, stream);
}

}  // extern "C"
