// layer_api.cpp -- C entry points of the decoder-layer operators: argument
// checks, then the launchers of layer.hpp.
#include <hip/hip_runtime.h>

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

// out: NormOut; the scale array's alignment and row length are the caller's.
qgemm_status norm_common(int out, const uint16_t *X, int64_t ldx, const uint16_t *R, int64_t ldr,
                         const uint16_t *gamma, float eps, uint16_t *Rout, int64_t ldo, void *Q, int64_t ldq, void *S,
                         int64_t lds, int64_t s_row, int64_t M, int64_t K, void *stream)
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
    if (M == 0)
        return QGEMM_OK;
    TRY(check_rows("X", X, ldx, K));
    if (R)
        TRY(check_rows("R", R, ldr, K));
    if (Rout)
        TRY(check_rows("Rout", Rout, ldo, K));
    TRY(check_rows("gamma", gamma, K, K));
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
    TRY(check_device());
    const NormArgs a = {X, R, gamma, Rout, (uint8_t *)Q, S, ldx, ldr, ldo, ldq, lds, (int)M, (int)K, eps};
    return launch([&] { return launch_rmsnorm_quant(out, a, (hipStream_t)stream); });
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

}  // extern "C"
