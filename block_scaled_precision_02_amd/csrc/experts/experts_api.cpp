// experts_api.cpp -- C entry points of the operators of a layer of experts:
// argument checks, then the launchers of experts.hpp.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../qgemm_host.hpp"
#include "../qgemm_kernel.hpp"
#include "../layer/layer.hpp"
#include "experts.hpp"

using namespace qgemm;

namespace {

constexpr int64_t MOE_MAX_SLOTS = (int64_t)1 << 30;

// bf16 rows of n elements, row stride ld elements.
qgemm_status check_rows(const char *name, const void *p, int64_t ld, int64_t n)
{
    if (!p)
        return fail(QGEMM_ERR_NULL_POINTER, "%s is NULL", name);
    if (!aligned(p, 16))
        return fail(QGEMM_ERR_BAD_LAYOUT, "%s is not 16-byte aligned", name);
    if (ld < n || ld % 8 || ld >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_LAYOUT, "row stride of %s, %lld elements: need >= %lld, a multiple of 8, below 2^31",
                    name, (long long)ld, (long long)n);
    return QGEMM_OK;
}

qgemm_status check_words(const char *name, const void *p)
{
    if (!p)
        return fail(QGEMM_ERR_NULL_POINTER, "%s is NULL", name);
    if (!aligned(p, 4))
        return fail(QGEMM_ERR_BAD_LAYOUT, "%s is not 4-byte aligned", name);
    return QGEMM_OK;
}

qgemm_status check_choices(int64_t tokens, int64_t top_k)
{
    if (tokens < 0 || top_k <= 0 || top_k > MOE_MAX_K || tokens >= MOE_MAX_SLOTS || tokens * top_k >= MOE_MAX_SLOTS)
        return fail(QGEMM_ERR_BAD_SHAPE, "tokens=%lld top_k=%lld: need tokens >= 0, top_k 1 to %d, tokens * top_k < 2^30",
                    (long long)tokens, (long long)top_k, MOE_MAX_K);
    return QGEMM_OK;
}

qgemm_status check_experts(int64_t experts)
{
    if (experts <= 0 || experts > MOE_MAX_EXPERTS)
        return fail(QGEMM_ERR_BAD_SHAPE, "experts=%lld: need 1 to %d", (long long)experts, MOE_MAX_EXPERTS);
    return QGEMM_OK;
}

qgemm_status check_exchange(int64_t tokens, int64_t top_k, int64_t rows, int64_t H)
{
    TRY(check_choices(tokens, top_k));
    if (rows < 0 || rows >= LD_LIMIT || H <= 0 || H % 8 || H >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_SHAPE, "rows=%lld H=%lld: need 0 <= rows < 2^31, H a positive multiple of 8 below 2^31",
                    (long long)rows, (long long)H);
    if (H / 8 > (int64_t)65535 * 256)
        return fail(QGEMM_ERR_BAD_SHAPE, "H=%lld is too large", (long long)H);
    return QGEMM_OK;
}

// out: NormOut; the scale array's alignment and row length are the caller's.
qgemm_status swiglu_common(int out, const uint16_t *X, int64_t ldx, const int32_t *count, void *Q, int64_t ldq, void *S,
                           int64_t lds, int64_t s_row, int64_t M, int64_t I, void *stream)
{
    if (M < 0 || I <= 0 || M >= LD_LIMIT || I >= LD_LIMIT / 2)
        return fail(QGEMM_ERR_BAD_SHAPE, "M=%lld I=%lld: need 0 <= M < 2^31, 0 < I < 2^30", (long long)M, (long long)I);
    const int64_t unit = out == NORM_F8_BLOCK ? 128 : 32;
    if (I % unit)
        return fail(QGEMM_ERR_BAD_SHAPE, "I=%lld is not a multiple of %lld", (long long)I, (long long)unit);
    if (!aligned(count, 4))
        return fail(QGEMM_ERR_BAD_LAYOUT, "count is not 4-byte aligned");
    if (M == 0)
        return QGEMM_OK;
    TRY(check_rows("X", X, ldx, 2 * I));
    if (!Q)
        return fail(QGEMM_ERR_NULL_POINTER, "Q is NULL");
    const int64_t q_row = out == NORM_MX_E2M1 ? I / 2 : I;
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
    TRY(check_device());
    const SwigluArgs a = {X, (uint8_t *)Q, S, count, ldx, ldq, lds, 0, (int)M, (int)I, 0, 0};
    return launch([&] { return launch_swiglu_quant(out, a, (hipStream_t)stream); });
}

qgemm_status grouped_common(int path, const void *A, int64_t lda, int64_t a_rows, const void *B, int64_t ldb,
                            const void *SA, const void *SB, const int32_t *offsets, const int32_t *order, int64_t top_k,
                            const uint16_t *bias, uint16_t *C, int64_t ldc, int64_t rows, int64_t experts, int64_t N,
                            int64_t K, void *stream)
{
    TRY(check_experts(experts));
    if (a_rows < 0 || rows < 0 || N < 0 || K <= 0 || a_rows >= LD_LIMIT || rows >= MOE_MAX_SLOTS || N >= LD_LIMIT ||
        K >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_SHAPE, "rows of A=%lld rows=%lld N=%lld K=%lld: need rows < 2^30, N < 2^31, K > 0",
                    (long long)a_rows, (long long)rows, (long long)N, (long long)K);
    if (K % 128)
        return fail(QGEMM_ERR_BAD_SHAPE, "K=%lld is not a multiple of 128", (long long)K);
    if (path == PATH_I8 && K > 131071)
        return fail(QGEMM_ERR_BAD_SHAPE, "K=%lld exceeds 131071 (int32 accumulator range)", (long long)K);
    if (top_k <= 0 || top_k > MOE_MAX_K)
        return fail(QGEMM_ERR_BAD_SHAPE, "top_k=%lld: need 1 to %d", (long long)top_k, MOE_MAX_K);
    if (!order && a_rows != rows)
        return fail(QGEMM_ERR_BAD_SHAPE, "without an order A has the rows themselves: %lld, not %lld", (long long)rows,
                    (long long)a_rows);
    if (rows == 0 || N == 0)
        return QGEMM_OK;
    if (a_rows == 0)
        return fail(QGEMM_ERR_BAD_SHAPE, "A has no rows");
    const int64_t kbytes = path == PATH_MX4 ? K / 2 : K;
    const struct { const char *name; const void *p; int64_t ld; } operands[] = {{"A", A, lda}, {"B", B, ldb}};
    for (const auto &o : operands) {
        if (!o.p)
            return fail(QGEMM_ERR_NULL_POINTER, "%s is NULL", o.name);
        if (!aligned(o.p, 16) || o.ld < kbytes || o.ld % 16 || o.ld * 256 >= LD_LIMIT)
            return fail(QGEMM_ERR_BAD_LAYOUT,
                        "%s must be 16-byte aligned with a row stride of %lld bytes >= %lld, a multiple of 16, 256 rows "
                        "below 2^31 bytes", o.name, (long long)o.ld, (long long)kbytes);
    }
    if (order && a_rows * lda >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_LAYOUT, "A of %lld rows of %lld bytes: with an order, need less than 2^31 bytes",
                    (long long)a_rows, (long long)lda);
    if (!SA || !SB)
        return fail(QGEMM_ERR_NULL_POINTER, "%s is NULL", SA ? "scale_b" : "scale_a");
    const unsigned sal = path == PATH_I8 || path == PATH_F8 ? 4 : 16;
    if (!aligned(SA, sal) || !aligned(SB, sal))
        return fail(QGEMM_ERR_BAD_LAYOUT, "scales must be %u-byte aligned", sal);
    if (!aligned(bias, 2))
        return fail(QGEMM_ERR_BAD_LAYOUT, "bias is not 2-byte aligned");
    if (!C)
        return fail(QGEMM_ERR_NULL_POINTER, "C is NULL");
    if (!aligned(C, 16) || ldc < N || ldc % 8 || ldc * 512 >= LD_LIMIT)
        return fail(QGEMM_ERR_BAD_LAYOUT,
                    "C must be 16-byte aligned with ldc=%lld >= N=%lld, a multiple of 8, 256 rows below 2^31 bytes",
                    (long long)ldc, (long long)N);
    TRY(check_words("offsets", offsets));
    if (!aligned(order, 4))
        return fail(QGEMM_ERR_BAD_LAYOUT, "order is not 4-byte aligned");
    const GroupedArgs a = {(const uint8_t *)A, (const uint8_t *)B, SA, SB, bias, C, offsets, order, lda, ldb, ldc,
                           ldb * N, a_rows, rows, (int)top_k, (int)experts, (int)N, (int)K};
    if (!grouped_fits(path, a))
        return fail(QGEMM_ERR_BAD_SHAPE, "rows=%lld, experts=%lld, N=%lld are too many for one call", (long long)rows,
                    (long long)experts, (long long)N);
    TRY(check_device());
    return launch([&] { return launch_grouped(path, a, (hipStream_t)stream); });
}

}  // namespace

extern "C" {

int64_t qgemm_moe_sort_workspace(int64_t tokens, int64_t top_k, int64_t experts)
{
    if (check_choices(tokens, top_k) != QGEMM_OK || check_experts(experts) != QGEMM_OK)
        return -1;
    SortArgs a = {};
    a.slots = (int)(tokens * top_k);
    a.experts = (int)experts;
    return sort_plan(a);
}

qgemm_status qgemm_moe_sort(const int32_t *ids, int64_t tokens, int64_t top_k, int64_t experts, int32_t *offsets,
                            int32_t *order, int32_t *position, void *workspace, int64_t workspace_bytes, void *stream)
{
    TRY(check_choices(tokens, top_k));
    TRY(check_experts(experts));
    TRY(check_words("offsets", offsets));
    SortArgs a = {};
    a.slots = (int)(tokens * top_k);
    a.experts = (int)experts;
    if (a.slots > 0) {
        TRY(check_words("ids", ids));
        TRY(check_words("order", order));
        TRY(check_words("position", position));
    }
    const int64_t need = sort_plan(a);
    if (need > 0) {
        if (!workspace)
            return fail(QGEMM_ERR_NULL_POINTER, "workspace is NULL; this call needs %lld bytes", (long long)need);
        if (!aligned(workspace, 16) || workspace_bytes < need)
            return fail(QGEMM_ERR_BAD_LAYOUT, "workspace of %lld bytes: need %lld, 16-byte aligned",
                        (long long)workspace_bytes, (long long)need);
    }
    TRY(check_device());
    a.ids = ids;
    a.offsets = offsets;
    a.order = order;
    a.position = position;
    a.hist = (int32_t *)workspace;
    return launch([&] { return launch_moe_sort(a, (hipStream_t)stream); });
}

qgemm_status qgemm_moe_gather(const uint16_t *X, int64_t ldx, const int32_t *position, uint16_t *Y, int64_t ldy,
                              int64_t tokens, int64_t top_k, int64_t rows, int64_t H, void *stream)
{
    TRY(check_exchange(tokens, top_k, rows, H));
    if (tokens == 0 || rows == 0)
        return QGEMM_OK;
    TRY(check_rows("X", X, ldx, H));
    TRY(check_rows("Y", Y, ldy, H));
    TRY(check_words("position", position));
    TRY(check_device());
    ExchangeArgs a = {};
    a.X = X;
    a.O = Y;
    a.position = position;
    a.ldx = ldx;
    a.ldo = ldy;
    a.rows = rows;
    a.tokens = (int)tokens;
    a.k = (int)top_k;
    a.H = (int)H;
    return launch([&] { return launch_moe_gather(a, (hipStream_t)stream); });
}

qgemm_status qgemm_moe_combine(const uint16_t *Y, int64_t ldy, const int32_t *position, const float *weights,
                               const uint16_t *R, int64_t ldr, uint16_t *O, int64_t ldo, int64_t tokens, int64_t top_k,
                               int64_t rows, int64_t H, void *stream)
{
    TRY(check_exchange(tokens, top_k, rows, H));
    if (tokens == 0)
        return QGEMM_OK;
    if (rows > 0)
        TRY(check_rows("Y", Y, ldy, H));
    if (R)
        TRY(check_rows("R", R, ldr, H));
    TRY(check_rows("O", O, ldo, H));
    TRY(check_words("position", position));
    if (!aligned(weights, 4))
        return fail(QGEMM_ERR_BAD_LAYOUT, "weights is not 4-byte aligned");
    TRY(check_device());
    ExchangeArgs a = {};
    a.X = R;
    a.Y = Y;
    a.O = O;
    a.W = weights;
    a.position = position;
    a.ldx = ldr;
    a.ldy = ldy;
    a.ldo = ldo;
    a.rows = rows;
    a.tokens = (int)tokens;
    a.k = (int)top_k;
    a.H = (int)H;
    return launch([&] { return launch_moe_combine(a, (hipStream_t)stream); });
}

qgemm_status qgemm_moe_combine_grad(const uint16_t *dO, int64_t lddo, const uint16_t *Y, int64_t ldy,
                                    const int32_t *position, const float *weights, uint16_t *dY, int64_t lddy,
                                    float *dweights, int64_t tokens, int64_t top_k, int64_t rows, int64_t H,
                                    void *stream)
{
    TRY(check_exchange(tokens, top_k, rows, H));
    if (tokens == 0)
        return QGEMM_OK;
    TRY(check_rows("dO", dO, lddo, H));
    if (rows > 0) {
        TRY(check_rows("Y", Y, ldy, H));
        TRY(check_rows("dY", dY, lddy, H));
    }
    TRY(check_words("position", position));
    TRY(check_words("weights", weights));
    TRY(check_words("dweights", dweights));
    TRY(check_device());
    ExchangeArgs a = {};
    a.X = dO;
    a.Y = Y;
    a.O = dY;
    a.W = weights;
    a.dW = dweights;
    a.position = position;
    a.ldx = lddo;
    a.ldy = ldy;
    a.ldo = lddy;
    a.rows = rows;
    a.tokens = (int)tokens;
    a.k = (int)top_k;
    a.H = (int)H;
    return launch([&] { return launch_moe_combine_grad(a, (hipStream_t)stream); });
}

qgemm_status qgemm_swiglu_quant_i8_rowwise(const uint16_t *X, int64_t ldx, const int32_t *count, int8_t *Q, int64_t ldq,
                                           float *scale, int64_t M, int64_t I, void *stream)
{
    return swiglu_common(NORM_I8_ROW, X, ldx, count, Q, ldq, scale, 0, 0, M, I, stream);
}

qgemm_status qgemm_swiglu_quant_f8_pertoken(const uint16_t *X, int64_t ldx, const int32_t *count, uint8_t *Q,
                                            int64_t ldq, float *scale, int64_t M, int64_t I, void *stream)
{
    return swiglu_common(NORM_F8_ROW, X, ldx, count, Q, ldq, scale, 0, 0, M, I, stream);
}

qgemm_status qgemm_swiglu_quant_f8_block(const uint16_t *X, int64_t ldx, const int32_t *count, uint8_t *Q, int64_t ldq,
                                         float *S, int64_t lds, int64_t M, int64_t I, void *stream)
{
    return swiglu_common(NORM_F8_BLOCK, X, ldx, count, Q, ldq, S, lds, I / 128, M, I, stream);
}

qgemm_status qgemm_swiglu_quant_mx(qgemm_mx_fmt fmt, const uint16_t *X, int64_t ldx, const int32_t *count, void *Q,
                                   int64_t ldq, uint8_t *S, int64_t lds, int64_t M, int64_t I, void *stream)
{
    if (fmt != QGEMM_MX_E4M3 && fmt != QGEMM_MX_E2M1)
        return fail(QGEMM_ERR_BAD_FORMAT, "unknown MX element format %d", (int)fmt);
    return swiglu_common(fmt == QGEMM_MX_E4M3 ? NORM_MX_E4M3 : NORM_MX_E2M1, X, ldx, count, Q, ldq, S, lds, I / 32, M,
                         I, stream);
}

qgemm_status qgemm_i8_rowwise_grouped(const int8_t *A, int64_t lda, int64_t a_rows, const int8_t *B, int64_t ldb,
                                      const float *scale_a, const float *scale_b, const int32_t *offsets,
                                      const int32_t *order, int64_t top_k, const uint16_t *bias, uint16_t *C,
                                      int64_t ldc, int64_t rows, int64_t experts, int64_t N, int64_t K, void *stream)
{
    return grouped_common(PATH_I8, A, lda, a_rows, B, ldb, scale_a, scale_b, offsets, order, top_k, bias, C, ldc, rows,
                          experts, N, K, stream);
}

qgemm_status qgemm_f8_pertoken_grouped(const uint8_t *A, int64_t lda, int64_t a_rows, const uint8_t *B, int64_t ldb,
                                       const float *scale_a, const float *scale_b, const int32_t *offsets,
                                       const int32_t *order, int64_t top_k, const uint16_t *bias, uint16_t *C,
                                       int64_t ldc, int64_t rows, int64_t experts, int64_t N, int64_t K, void *stream)
{
    return grouped_common(PATH_F8, A, lda, a_rows, B, ldb, scale_a, scale_b, offsets, order, top_k, bias, C, ldc, rows,
                          experts, N, K, stream);
}

qgemm_status qgemm_f8_blockscale_grouped(const uint8_t *A, int64_t lda, int64_t a_rows, const uint8_t *B, int64_t ldb,
                                         const float *scale_a, const float *scale_b, const int32_t *offsets,
                                         const int32_t *order, int64_t top_k, const uint16_t *bias, uint16_t *C,
                                         int64_t ldc, int64_t rows, int64_t experts, int64_t N, int64_t K,
                                         void *stream)
{
    return grouped_common(PATH_F8B, A, lda, a_rows, B, ldb, scale_a, scale_b, offsets, order, top_k, bias, C, ldc, rows,
                          experts, N, K, stream);
}

qgemm_status qgemm_mx_grouped(qgemm_mx_fmt fmt, const void *A, int64_t lda, int64_t a_rows, const void *B, int64_t ldb,
                              const uint8_t *scale_a, const uint8_t *scale_b, const int32_t *offsets,
                              const int32_t *order, int64_t top_k, const uint16_t *bias, uint16_t *C, int64_t ldc,
                              int64_t rows, int64_t experts, int64_t N, int64_t K, void *stream)
{
    if (fmt != QGEMM_MX_E4M3 && fmt != QGEMM_MX_E2M1)
        return fail(QGEMM_ERR_BAD_FORMAT, "MX element format %d: need e4m3 or e2m1", (int)fmt);
    return grouped_common(fmt == QGEMM_MX_E4M3 ? PATH_MX8 : PATH_MX4, A, lda, a_rows, B, ldb, scale_a, scale_b, offsets,
                          order, top_k, bias, C, ldc, rows, experts, N, K, stream);
}

int qgemm_select_grouped_tile(int path, int64_t rows, int64_t experts, int64_t N)
{
    if (path < PATH_I8 || path > PATH_F8B || rows <= 0 || rows >= MOE_MAX_SLOTS || experts <= 0 ||
        experts > MOE_MAX_EXPERTS || N <= 0 || N >= LD_LIMIT)
        return -1;
    GroupedArgs a = {};
    a.rows = rows;
    a.experts = (int)experts;
    a.N = (int)N;
    return grouped_tile_id(path, a);
}

}  // extern "C"
