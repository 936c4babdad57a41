// C ABI of the products with 4-bit weights: plan creation and validation, kernel choice, launch.
// Host code only; the kernels live in gemm_quant.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/gemm.h"
#include "gemm_internal.h"
#include "host_common.h"

using namespace tge::host;
using tge::QuantEntry;
using tge::QuantParams;

struct gemm_quant_plan {
    int64_t rows, N, K, block, groups;
    int64_t lda, ldq, lds, ldc, stride_q, stride_s, stride_bias;
    int ab, cd, epi;
    bool zeros;
    const QuantEntry *kernel;
    char desc[256];
};

namespace {

constexpr int64_t MAX_K = (int64_t)1 << 23;   // 2^16 chunks of 128 (see block_of in gemm_quant.hip)

using RowsFn = const QuantEntry *(*)(int, int);
using TileFn = const QuantEntry *(*)(int);

RowsFn rows_table(int ab, int cd) {
    if (ab == GEMM_F16 && cd == GEMM_F16) return tge::quant_rows_f16_f16;
    if (ab == GEMM_F16 && cd == GEMM_F32) return tge::quant_rows_f16_f32;
    if (ab == GEMM_BF16 && cd == GEMM_BF16) return tge::quant_rows_bf16_bf16;
    if (ab == GEMM_BF16 && cd == GEMM_F32) return tge::quant_rows_bf16_f32;
    return nullptr;
}

TileFn tile_table(int ab, int cd) {
    if (ab == GEMM_F16 && cd == GEMM_F16) return tge::quant_tile_f16_f16;
    if (ab == GEMM_F16 && cd == GEMM_F32) return tge::quant_tile_f16_f32;
    if (ab == GEMM_BF16 && cd == GEMM_BF16) return tge::quant_tile_bf16_bf16;
    if (ab == GEMM_BF16 && cd == GEMM_F32) return tge::quant_tile_bf16_f32;
    return nullptr;
}

// Workgroups of a launch; by expert, enough for any split of the rows over the experts.
int64_t grid_of(const gemm_quant_plan &p, bool by_expert) {
    const int64_t tm = by_expert ? row_tiles(p.rows, p.groups, p.kernel->bm) : ceil_div(p.rows, p.kernel->bm);
    return tm * ceil_div(p.N, p.kernel->bn);
}

// Whether the 128 x 128 tiles beat the kernel for few rows (16 x 64).  Both take a time in
// proportion to K; at K = 4096 a round of tiles takes 58 to 79 us however few there are and 0.19 us per
// tile from two per CU on (blocks of 32: 88 to 102, and 0.25), the other kernel 0.022 to 0.045 us per
// workgroup, by type, block and zero points.  Measured (few rows -> tiles): bf16, blocks of 128 without
// zero points, 512 x 4096 x 4096 62 vs 69 us, 700 rows 78 -> 68, 1024 113 -> 70, 2048 x 1024 x 4096 57 vs 68,
// 256 x 16384 x 2048 64 -> 39, 512 x 8192 x 8192 192 -> 129; with zero points 512 x 4096 x 4096 74 -> 58,
// 256 rows 40 vs 58; 600 rows, blocks of 64 75 vs 74 without them and 95 -> 79 with, blocks of 32
// 97 vs 92 and 111 -> 102.  fp16, 700 rows: blocks of 128 69 -> 67 and 90 -> 65, of 64 77 -> 71 and
// 94 -> 75, of 32 79 vs 88 and 108 -> 97.  Experts' ranges end inside a tile: half a tile each is counted.
bool tiles_pay(const gemm_quant_plan &p) {
    static const double few_us[2][3][2] = {{{0.031, 0.037}, {0.027, 0.032}, {0.022, 0.030}},    // [bf16][block][zeros]
                                           {{0.038, 0.045}, {0.029, 0.038}, {0.028, 0.037}}};
    const double ragged = p.groups > 1 ? 0.5 * (double)(p.rows < p.groups ? p.rows : p.groups) : 0.0;
    const double few = ((double)p.rows / 16 + ragged) * (double)ceil_div(p.N, 64);
    const double tiles = ((double)p.rows / 128 + ragged) * (double)ceil_div(p.N, 128);
    const double round = p.block == 32 ? 95.0 : 70.0, t = (p.block == 32 ? 0.25 : 0.19) * tiles;
    return few_us[p.ab == GEMM_BF16][p.block == 32 ? 0 : p.block == 64 ? 1 : 2][p.zeros != 0] * few > (t > round ? t : round);
}

}  // namespace

extern "C" {

gemm_status_t gemm_quant_plan_create(gemm_quant_plan_t *out, const gemm_quant_desc_t *d) {
    if (!out) return GEMM_STATUS_INVALID_VALUE;
    *out = nullptr;
    if (!d) return GEMM_STATUS_INVALID_VALUE;
    const int ab = bits(d->ab_type), cd = bits(d->cd_type), epi = bits(d->epilogue), algo = bits(d->algo),
              tile = d->tile;
    if (!in(ab, GEMM_F32, GEMM_DF32) || !in(cd, GEMM_F32, GEMM_DF32) || !in(epi, GEMM_EPI_NONE, GEMM_EPI_BIAS_RELU) ||
        !in(d->zeros, 0, 1))
        return GEMM_STATUS_INVALID_VALUE;
    switch (algo) {
    case GEMM_ALGO_AUTO: if (tile != 0) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_FAST: if (tile != 0 && tile != 128) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_SKINNY:
        if (tile != 0 && tile != 16 && tile != 64) return GEMM_STATUS_INVALID_VALUE;
        break;
    default: return GEMM_STATUS_INVALID_VALUE;
    }
    if (d->rows < 0 || d->N < 0 || d->K < 0 || d->groups < 1 || d->block < 1 || d->K % d->block != 0)
        return GEMM_STATUS_INVALID_VALUE;
    if (!rows_table(ab, cd) || !(d->block == 32 || d->block == 64 || d->block % 128 == 0))
        return GEMM_STATUS_NOT_SUPPORTED;
    if (d->rows >= LIM31 || d->N >= LIM31 || d->K >= MAX_K || d->lda >= LIM31 || d->ldq >= LIM31 ||
        d->lds >= LIM31 || d->ldc >= LIM31 || d->groups >= MAX_GROUPS)
        return GEMM_STATUS_NOT_SUPPORTED;
    const int64_t nb = d->K / d->block;
    if (d->lda < (d->K > 1 ? d->K : 1) || d->ldq < d->K / 2 || d->lds < nb || d->ldc < (d->N > 1 ? d->N : 1) ||
        d->stride_q < 0 || d->stride_s < 0 || d->stride_bias < 0)
        return GEMM_STATUS_INVALID_VALUE;
    const int64_t big = ((int64_t)1 << 62) / 8 / d->groups;
    if (d->stride_q > big || d->stride_s > big || d->stride_bias > big) return GEMM_STATUS_NOT_SUPPORTED;

    gemm_quant_plan p = {};
    p.rows = d->rows; p.N = d->N; p.K = d->K; p.block = d->block; p.groups = d->groups;
    p.lda = d->lda; p.ldq = d->ldq; p.lds = d->lds; p.ldc = d->ldc;
    p.stride_q = d->stride_q; p.stride_s = d->stride_s; p.stride_bias = d->stride_bias;
    p.ab = ab; p.cd = cd; p.epi = epi; p.zeros = d->zeros != 0;
    const int g = d->block >= 128 ? 128 : (int)d->block;
    // rows kernels: the wide one where it still gives every CU a workgroup
    const auto rows_kernel = [&]() {
        p.kernel = rows_table(ab, cd)(g, 4);
        return grid_of(p, p.groups > 1) >= 256 ? p.kernel : rows_table(ab, cd)(g, 1);
    };
    if (algo == GEMM_ALGO_SKINNY) p.kernel = tile ? rows_table(ab, cd)(g, tile / 16) : rows_kernel();
    else if (algo == GEMM_ALGO_FAST) p.kernel = tile_table(ab, cd)(g);
    else p.kernel = tiles_pay(p) ? tile_table(ab, cd)(g) : rows_kernel();
    if (grid_of(p, true) >= MAX_GRID) return GEMM_STATUS_NOT_SUPPORTED;
    gemm_quant_plan *q = new (std::nothrow) gemm_quant_plan(p);
    if (!q) return GEMM_STATUS_ALLOC_FAILED;
    snprintf(q->desc, sizeof q->desc, "%s %s->%s block %lld%s tile %dx%d groups %lld grid %lld", p.kernel->name,
             type_name(ab), type_name(cd), (long long)p.block, p.zeros ? " zeros" : "", p.kernel->bm, p.kernel->bn,
             (long long)p.groups, (long long)grid_of(p, p.groups > 1));
    *out = q;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_quant_run(gemm_quant_plan_t p, const void *A, const void *Q, const void *scales,
                             const void *zeros, const void *C, void *D, const void *bias,
                             const int32_t *offsets, float alpha, float beta, void *stream) {
    if (!p) return GEMM_STATUS_INVALID_VALUE;
    if (p->rows == 0 || p->N == 0) return GEMM_STATUS_SUCCESS;
    if (alpha != alpha || beta != beta) return GEMM_STATUS_INVALID_VALUE;   // NaN scalars
    const int ecd = elem_bytes(p->cd);
    const bool has_bias = p->epi == GEMM_EPI_BIAS || p->epi == GEMM_EPI_BIAS_RELU;
    if (!D || !aligned(D, ecd)) return GEMM_STATUS_INVALID_VALUE;
    if (p->K > 0 && (!A || !Q || !scales || !aligned(A, 2) || !aligned(scales, 2) || (p->zeros && !zeros)))
        return GEMM_STATUS_INVALID_VALUE;
    if (beta != 0.0f && (!C || !aligned(C, ecd))) return GEMM_STATUS_INVALID_VALUE;
    if (has_bias && (!bias || !aligned(bias, 4))) return GEMM_STATUS_INVALID_VALUE;
    if (offsets ? !aligned(offsets, 4) : p->groups > 1) return GEMM_STATUS_INVALID_VALUE;
    QuantParams prm = {};
    prm.A = A; prm.C = C; prm.D = D; prm.bias = has_bias ? bias : nullptr;
    prm.M = (int)p->rows; prm.N = (int)p->N; prm.K = (int)p->K;
    prm.lda = (int)p->lda; prm.ldc = (int)p->ldc;
    prm.alpha = alpha; prm.beta = beta;
    prm.has_beta = beta != 0.0f;
    prm.has_bias = has_bias;
    prm.relu = p->epi == GEMM_EPI_RELU || p->epi == GEMM_EPI_BIAS_RELU;
    prm.tiles_m = (int)ceil_div(p->rows, p->kernel->bm);
    prm.tiles_n = (int)ceil_div(p->N, p->kernel->bn);
    prm.group_m = GROUP_M;
    prm.stride_bias = p->stride_bias;
    prm.offs = offsets;
    prm.groups = (int)p->groups;
    prm.rows = (int)p->rows;
    prm.Q = static_cast<const uint8_t *>(Q);
    prm.scales = scales;
    prm.zeros = p->zeros ? static_cast<const uint8_t *>(zeros) : nullptr;
    prm.stride_q = p->stride_q; prm.stride_s = p->stride_s;
    prm.ldq = (int)p->ldq; prm.lds = (int)p->lds; prm.block = (int)p->block;
    if (p->block >= 128) prm.block_rcp = (((uint64_t)1 << 32) + p->block / 128 - 1) / (p->block / 128);
    const unsigned grid = (unsigned)grid_of(*p, offsets != nullptr);
    return p->kernel->launch(prm, grid, static_cast<hipStream_t>(stream)) == hipSuccess ? GEMM_STATUS_SUCCESS
                                                                                       : GEMM_STATUS_HIP_ERROR;
}

gemm_status_t gemm_quant_plan_destroy(gemm_quant_plan_t p) {
    delete p;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_quant_plan_describe(gemm_quant_plan_t p, char *buf, size_t len) {
    if (!p || !buf || len == 0) return GEMM_STATUS_INVALID_VALUE;
    snprintf(buf, len, "%s", p->desc);
    return GEMM_STATUS_SUCCESS;
}

}  // extern "C"
