// C ABI of layer norm and its gradients: plan creation and validation, launch.  Host code only; the
// kernels are in layer_norm.hip.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/gemm.h"
#include "gemm_internal.h"
#include "host_common.h"

using namespace tge::host;
using tge::NormParams;
using tge::NormShape;

struct gemm_norm_plan {
    int64_t rows, N, ldx, ldy;
    int type;
    float eps;
    NormShape forward, grad;
    int64_t grid_forward;              // workgroups
    int64_t grid_grad, grid_rows;      // the gradient's: with column sums (a partial sum each), and without
    size_t workspace;
    char desc[256];
};

namespace {

constexpr int64_t MAX_ROW_BYTES = 65536;

using RunFn = hipError_t (*)(const NormParams &, NormShape, unsigned, hipStream_t);

RunFn forward_of(int t) {
    return t == GEMM_F32 ? tge::norm_forward_f32 : t == GEMM_F16 ? tge::norm_forward_f16 : tge::norm_forward_bf16;
}
RunFn grad_of(int t) {
    return t == GEMM_F32 ? tge::norm_grad_f32 : t == GEMM_F16 ? tge::norm_grad_f16 : tge::norm_grad_bf16;
}

NormParams params(const gemm_norm_plan &p) {
    NormParams q = {};
    q.rows = (int)p.rows; q.N = (int)p.N; q.ldx = (int)p.ldx; q.ldy = (int)p.ldy;
    q.eps = p.eps;
    q.rn = 1.0f / (float)p.N;
    return q;
}

bool bad(const void *p, int to, bool required) { return p ? !aligned(p, (uintptr_t)to) : required; }

}  // namespace

extern "C" {

gemm_status_t gemm_norm_plan_create(gemm_norm_plan_t *out, const gemm_norm_desc_t *d) {
    if (!out) return GEMM_STATUS_INVALID_VALUE;
    *out = nullptr;
    if (!d) return GEMM_STATUS_INVALID_VALUE;
    const int type = bits(d->type);
    if (!in(type, GEMM_F32, GEMM_DF32) || d->rows < 0 || d->N < 0 || !(d->eps >= 0.0f) || isinf(d->eps))
        return GEMM_STATUS_INVALID_VALUE;
    if (d->ldx < (d->N > 1 ? d->N : 1) || d->ldy < (d->N > 1 ? d->N : 1)) return GEMM_STATUS_INVALID_VALUE;
    if (type > GEMM_BF16) return GEMM_STATUS_NOT_SUPPORTED;
    const int es = elem_bytes(type);
    // the kernels step over the rows by less than 2^20 in 32 bits
    if (d->rows >= LIM31 - (1 << 20) || d->N > MAX_ROW_BYTES / es || d->ldx >= LIM31 || d->ldy >= LIM31)
        return GEMM_STATUS_NOT_SUPPORTED;
    gemm_norm_plan p = {};
    p.rows = d->rows; p.N = d->N; p.ldx = d->ldx; p.ldy = d->ldy;
    p.type = type;
    p.eps = d->eps;
    const int64_t pieces = d->N > 0 ? ceil_div(d->N * es, 16) : 1;
    p.forward = tge::norm_shape(pieces, false);
    p.grad = tge::norm_shape(pieces, true);
    // as many workgroups as the chip holds at once, each with rows enough to keep the next one's loads
    // in flight
    const int64_t fw = p.forward.waves * p.forward.teams;
    const int64_t most_f = 256 * (16 / fw > 1 ? 16 / fw : 1);
    const int64_t side = 64 / p.forward.lanes;       // rows of a team
    const int64_t need_f = ceil_div(d->rows, p.forward.teams * side), need_g = ceil_div(d->rows, p.grad.teams * side);
    p.grid_forward = need_f < most_f ? need_f : most_f;
    // The gradient's write and join a partial sum each, 16 N bytes moved at some 5 TB/s, against 3 us for each turn
    // of rows that others do not take: the least of both together, at most one to a CU.  us by workgroups: 300
    // rows of 16384 64 24.5, 133 20.8; 1200 rows of 8192 180 23.7, 256 20.5; 60 rows of 4096 30 7.5, 15 8.8
    const double both = sqrt((double)need_g * 3e-6 * 5e12 / (16.0 * (double)(d->N > 1 ? d->N : 1)));
    const int64_t most_g = both < 256.0 ? (int64_t)both + 1 : 256;
    p.grid_grad = need_g < most_g ? need_g : most_g;
    p.grid_rows = need_g < 256 ? need_g : 256;
    p.workspace = (size_t)(p.grid_grad * 2 * d->N * 4);
    gemm_norm_plan *q = new (std::nothrow) gemm_norm_plan(p);
    if (!q) return GEMM_STATUS_ALLOC_FAILED;
    snprintf(q->desc, sizeof q->desc, "norm %s N %lld waves %d chunks %d grid %lld, gradient %lld", type_name(type),
             (long long)p.N, p.forward.waves, p.forward.chunks, (long long)p.grid_forward, (long long)p.grid_grad);
    *out = q;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_norm_workspace_bytes(gemm_norm_plan_t p, size_t *bytes) {
    if (!p || !bytes) return GEMM_STATUS_INVALID_VALUE;
    *bytes = p->workspace;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_norm_run(gemm_norm_plan_t p, const void *X, const float *weight, const float *bias, void *Y,
                            float *mean, float *rstd, void *stream) {
    if (!p) return GEMM_STATUS_INVALID_VALUE;
    if (p->rows == 0 || p->N == 0) return GEMM_STATUS_SUCCESS;
    const int es = elem_bytes(p->type);
    if (bad(X, es, true) || bad(Y, es, true) || bad(weight, 4, false) || bad(bias, 4, false) ||
        bad(mean, 4, false) || bad(rstd, 4, false))
        return GEMM_STATUS_INVALID_VALUE;
    NormParams q = params(*p);
    q.X = X; q.weight = weight; q.bias = bias; q.Y = Y; q.mean = mean; q.rstd = rstd;
    return forward_of(p->type)(q, p->forward, (unsigned)p->grid_forward, static_cast<hipStream_t>(stream)) == hipSuccess
               ? GEMM_STATUS_SUCCESS
               : GEMM_STATUS_HIP_ERROR;
}

gemm_status_t gemm_norm_grad_run(gemm_norm_plan_t p, const void *dY, const void *X, const float *weight,
                                 const float *mean, const float *rstd, const void *C, void *dX, float *dweight,
                                 float *dbias, float beta, void *workspace, size_t workspace_bytes, void *stream) {
    if (!p || beta != beta) return GEMM_STATUS_INVALID_VALUE;
    if (p->N == 0) return GEMM_STATUS_SUCCESS;
    const bool sums = dweight || dbias, has_rows = p->rows > 0;
    const int es = elem_bytes(p->type);
    if (bad(dY, es, has_rows) || bad(X, es, has_rows) || bad(dX, es, has_rows) || bad(weight, 4, false) ||
        bad(mean, 4, has_rows) || bad(rstd, 4, has_rows) || bad(C, es, has_rows && beta != 0.0f) ||
        bad(dweight, 4, false) || bad(dbias, 4, false))
        return GEMM_STATUS_INVALID_VALUE;
    if (sums && has_rows && (bad(workspace, 4, true) || workspace_bytes < p->workspace)) return GEMM_STATUS_INVALID_VALUE;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    float *part = sums && has_rows ? static_cast<float *>(workspace) : nullptr;
    if (has_rows) {
        NormParams q = params(*p);
        q.X = X; q.weight = weight; q.Y = const_cast<void *>(dY);
        q.mean = const_cast<float *>(mean); q.rstd = const_cast<float *>(rstd);
        q.C = C; q.dX = dX;
        q.part = part;
        q.beta = beta;
        q.has_beta = beta != 0.0f;
        const int64_t grid = sums ? p->grid_grad : p->grid_rows;
        if (grad_of(p->type)(q, p->grad, (unsigned)grid, st) != hipSuccess) return GEMM_STATUS_HIP_ERROR;
    }
    // without rows the sums are 0
    if (sums && tge::norm_join(part, has_rows ? (int)p->grid_grad : 0, (int)p->N, dweight, dbias, st) != hipSuccess)
        return GEMM_STATUS_HIP_ERROR;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_norm_plan_destroy(gemm_norm_plan_t p) {
    delete p;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_norm_plan_describe(gemm_norm_plan_t p, char *buf, size_t len) {
    if (!p || !buf || len == 0) return GEMM_STATUS_INVALID_VALUE;
    snprintf(buf, len, "%s", p->desc);
    return GEMM_STATUS_SUCCESS;
}

}  // extern "C"
