// C ABI of the routing of rows to experts and its gradient: plan creation and validation, launch.
// Host code only; the kernels are in route.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/gemm.h"
#include "gemm_internal.h"
#include "host_common.h"

using namespace tge::host;
using tge::RouteParams;
using tge::RouteShape;

struct gemm_route_plan {
    int64_t rows, experts, k, ldl;
    int type, normalize;
    RouteShape shape;
    int64_t block_rows, blocks, stride, grid_grad;
    size_t workspace;
    char desc[256];
};

namespace {

using ChooseFn = hipError_t (*)(const RouteParams &, RouteShape, hipStream_t);
using GradFn = hipError_t (*)(const RouteParams &, RouteShape, unsigned, hipStream_t);

ChooseFn choose_of(int t) {
    return t == GEMM_F32 ? tge::route_choose_f32 : t == GEMM_F16 ? tge::route_choose_f16 : tge::route_choose_bf16;
}
GradFn grad_of(int t) {
    return t == GEMM_F32 ? tge::route_grad_f32 : t == GEMM_F16 ? tge::route_grad_f16 : tge::route_grad_bf16;
}

// Lanes of a row and experts per lane: 16 lanes while 8 experts each are enough (their moves need no
// LDS), then wider.
RouteShape shape_of(int64_t experts) {
    static const RouteShape shapes[] = {{16, 1}, {16, 2}, {16, 4}, {16, 8}, {32, 8}, {64, 8}, {64, 16}};
    for (const RouteShape &s : shapes)
        if (experts <= s.lanes * s.per) return s;
    return {0, 0};
}

RouteParams params(const gemm_route_plan &p) {
    RouteParams q = {};
    q.rows = (int)p.rows; q.experts = (int)p.experts; q.k = (int)p.k; q.ldl = (int)p.ldl;
    q.normalize = p.normalize;
    q.block_rows = (int)p.block_rows;
    q.blocks = (int)p.blocks;
    q.stride = (int)p.stride;
    return q;
}

bool bad(const void *p, int to, bool required) { return p ? !aligned(p, (uintptr_t)to) : required; }

}  // namespace

extern "C" {

gemm_status_t gemm_route_plan_create(gemm_route_plan_t *out, const gemm_route_desc_t *d) {
    if (!out) return GEMM_STATUS_INVALID_VALUE;
    *out = nullptr;
    if (!d) return GEMM_STATUS_INVALID_VALUE;
    const int type = bits(d->type);
    if (!in(type, GEMM_F32, GEMM_DF32) || d->rows < 0 || d->experts < 1 || d->k < 1 || d->k > d->experts ||
        d->ldl < d->experts || !in(d->normalize, 0, 1))
        return GEMM_STATUS_INVALID_VALUE;
    if (type > GEMM_BF16 || d->experts > tge::ROUTE_MAX_EXPERTS || d->k > tge::ROUTE_MAX_K || d->ldl >= LIM31 ||
        d->rows >= LIM31 - (1 << 20) || d->rows * d->k >= LIM31 - (1 << 20))
        return GEMM_STATUS_NOT_SUPPORTED;
    gemm_route_plan p = {};
    p.rows = d->rows; p.experts = d->experts; p.k = d->k; p.ldl = d->ldl;
    p.type = type; p.normalize = d->normalize;
    p.shape = shape_of(d->experts);
    const int waves = tge::route_waves(p.shape.lanes * p.shape.per);
    const int64_t slots = waves * (64 / p.shape.lanes);    // rows that a workgroup chooses for at a time
    // one workgroup does a few rows in one launch; more take two, with up to ROUTE_MAX_BLOCKS workgroups
    const int64_t fill = ceil_div(ceil_div(d->rows, tge::ROUTE_MAX_BLOCKS), slots) * slots;
    const int64_t one = tge::route_one_rows(waves, p.shape.lanes);
    p.block_rows = d->rows <= one ? one : fill;
    p.blocks = d->rows > 0 ? ceil_div(d->rows, p.block_rows) : 1;
    const int64_t need = ceil_div(d->rows, 4 * (64 / p.shape.lanes));
    p.grid_grad = need < 2048 ? need : 2048;
    p.stride = 4;
    while (p.stride < p.blocks) p.stride *= 2;
    p.workspace = p.blocks > 1 ? (size_t)((2 * p.experts + 1) * p.stride * 4) : 0;
    gemm_route_plan *q = new (std::nothrow) gemm_route_plan(p);
    if (!q) return GEMM_STATUS_ALLOC_FAILED;
    snprintf(q->desc, sizeof q->desc, "route %s experts %lld k %lld%s lanes %d x %d blocks %lld of %lld rows", type_name(type),
             (long long)p.experts, (long long)p.k, p.normalize ? " normalized" : "", p.shape.lanes, p.shape.per,
             (long long)p.blocks, (long long)p.block_rows);
    *out = q;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_route_workspace_bytes(gemm_route_plan_t p, size_t *bytes) {
    if (!p || !bytes) return GEMM_STATUS_INVALID_VALUE;
    *bytes = p->workspace;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_route_run(gemm_route_plan_t p, const void *logits, const uint8_t *mask, int32_t *index,
                             float *weight, int32_t *order, int32_t *place, int32_t *offsets, float *slope,
                             float *loss, void *workspace, size_t workspace_bytes, void *stream) {
    if (!p) return GEMM_STATUS_INVALID_VALUE;
    const bool has_rows = p->rows > 0;
    if (bad(logits, elem_bytes(p->type), has_rows) || bad(index, 4, has_rows) || bad(weight, 4, has_rows) ||
        bad(order, 4, has_rows) || bad(place, 4, has_rows) || bad(offsets, 4, true) || bad(slope, 4, false) ||
        bad(loss, 4, false))
        return GEMM_STATUS_INVALID_VALUE;
    if (p->workspace && (bad(workspace, 4, true) || workspace_bytes < p->workspace)) return GEMM_STATUS_INVALID_VALUE;
    RouteParams q = params(*p);
    q.logits = logits; q.mask = mask; q.index = index; q.weight = weight; q.order = order; q.place = place;
    q.offsets = offsets; q.slope = slope; q.loss = loss;
    if (p->blocks > 1) {
        q.hist = static_cast<int32_t *>(workspace);
        q.psum = reinterpret_cast<float *>(q.hist + (p->experts + 1) * p->stride);
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (choose_of(p->type)(q, p->shape, st) != hipSuccess) return GEMM_STATUS_HIP_ERROR;
    if (p->blocks > 1 && tge::route_place(q, st) != hipSuccess) return GEMM_STATUS_HIP_ERROR;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_route_grad_run(gemm_route_plan_t p, const void *logits, const uint8_t *mask, const int32_t *index,
                                  const float *dweight, const float *slope, const float *dloss, void *dlogits,
                                  void *stream) {
    if (!p) return GEMM_STATUS_INVALID_VALUE;
    if (p->rows == 0) return GEMM_STATUS_SUCCESS;
    const int es = elem_bytes(p->type);
    if (bad(logits, es, true) || bad(dlogits, es, true) || bad(index, 4, dweight != nullptr) || bad(dweight, 4, false) ||
        bad(dloss, 4, false) || bad(slope, 4, dloss != nullptr))
        return GEMM_STATUS_INVALID_VALUE;
    RouteParams q = params(*p);
    q.logits = logits; q.mask = mask; q.index = const_cast<int32_t *>(index); q.dweight = dweight;
    q.slope = const_cast<float *>(slope); q.dloss = dloss; q.dlogits = dlogits;
    return grad_of(p->type)(q, p->shape, (unsigned)p->grid_grad, static_cast<hipStream_t>(stream)) == hipSuccess
               ? GEMM_STATUS_SUCCESS
               : GEMM_STATUS_HIP_ERROR;
}

gemm_status_t gemm_route_plan_destroy(gemm_route_plan_t p) {
    delete p;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_route_plan_describe(gemm_route_plan_t p, char *buf, size_t len) {
    if (!p || !buf || len == 0) return GEMM_STATUS_INVALID_VALUE;
    snprintf(buf, len, "%s", p->desc);
    return GEMM_STATUS_SUCCESS;
}

}  // extern "C"
