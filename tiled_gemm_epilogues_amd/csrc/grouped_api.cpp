// C ABI of the products grouped by expert: plan creation and validation, kernel choice, launch.
// Host code only; the kernels are the grouped instances of gemm_kernels.hip and gemm_fast.hip, and
// gemm_rows16.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/gemm.h"
#include "gemm_internal.h"
#include "host_common.h"

using namespace tge::host;
using tge::GroupedEntry;
using tge::GroupedParams;

struct gemm_grouped_plan {
    int mode;                        // tge::GROUP_ROWS or GROUP_K
    int64_t rows, M, N, K, groups;   // K unused by GROUP_K, M by GROUP_ROWS
    int64_t lda, ldb, ldc, stride_b, stride_bias, stride_c;
    int ab, cd, epi;
    const GroupedEntry *any;         // the kernel for any alignment: general, register-staged or for few rows
    const GroupedEntry *fast;        // aligned pointers: the fast kernel with direct loads, else nullptr
    char desc[256];
};

namespace {

constexpr int64_t FAST_MIN_K = 64;         // one slab of the fast kernel (16-bit inputs)
// Rows of a gradient plan, at most: the kernels add a step of up to 256 to a row number in 32 bits.
constexpr int64_t MAX_SUM_ROWS = LIM31 - 1024;

using TableFn = const GroupedEntry *(*)(int, int, int);
using FastFn = const GroupedEntry *(*)(int, int, int, int);
using RowsFn = const GroupedEntry *(*)(int, int);

TableFn any_table(int ab, int cd) {
    if (ab == GEMM_F32 && cd == GEMM_F32) return tge::grouped_any_f32_f32;
    if (ab == GEMM_F16 && cd == GEMM_F16) return tge::grouped_any_f16_f16;
    if (ab == GEMM_F16 && cd == GEMM_F32) return tge::grouped_any_f16_f32;
    if (ab == GEMM_BF16 && cd == GEMM_BF16) return tge::grouped_any_bf16_bf16;
    if (ab == GEMM_BF16 && cd == GEMM_F32) return tge::grouped_any_bf16_f32;
    return nullptr;
}

FastFn fast_table(int ab, int cd) {
    if (ab == GEMM_F16) return cd == GEMM_F16 ? tge::grouped_fast_f16_f16 : tge::grouped_fast_f16_f32;
    if (ab == GEMM_BF16) return cd == GEMM_BF16 ? tge::grouped_fast_bf16_bf16 : tge::grouped_fast_bf16_f32;
    return nullptr;
}

// Workgroups of a launch, at most MAX_GRID.
int64_t grid_of(const gemm_grouped_plan &p, const GroupedEntry &k, bool colsum) {
    const int64_t tn = ceil_div(p.N, k.bn);
    const __int128 g = p.mode == tge::GROUP_ROWS
                           ? (__int128)row_tiles(p.rows, p.groups, k.bm) * tn
                           : (__int128)p.groups * (ceil_div(p.M, k.bm) * tn + (colsum ? ceil_div(p.N, tge::COLSUM_COLS) : 0));
    return g < MAX_GRID ? (int64_t)g : MAX_GRID;
}

// What both descriptions have in common: ranges, types, algorithm.  SUCCESS when they hold.
gemm_status_t check_common(int64_t rows, int64_t N, int64_t MK, int64_t groups, int64_t lda, int64_t ldb,
                           int64_t ldc, int ab, int cd) {
    if (rows < 0 || N < 0 || MK < 0 || groups < 1) return GEMM_STATUS_INVALID_VALUE;
    if (rows >= LIM31 || N >= LIM31 || MK >= LIM31 || lda >= LIM31 || ldb >= LIM31 || ldc >= LIM31 ||
        groups >= MAX_GROUPS)
        return GEMM_STATUS_NOT_SUPPORTED;
    return any_table(ab, cd) ? GEMM_STATUS_SUCCESS : GEMM_STATUS_NOT_SUPPORTED;
}

// The launch of either mode; the arguments have been checked.
gemm_status_t launch(const gemm_grouped_plan &p, const void *A, const void *B, const void *C, void *D,
                     const void *bias, float *colsum, const int32_t *offsets, float alpha, float beta,
                     void *stream) {
    GroupedParams prm = {};
    prm.A = A; prm.B = B; prm.C = C; prm.D = D; prm.bias = bias;
    prm.M = (int)p.M; prm.N = (int)p.N; prm.K = (int)p.K;
    prm.lda = (int)p.lda; prm.ldb = (int)p.ldb; prm.ldc = (int)p.ldc;
    prm.alpha = alpha; prm.beta = beta;
    prm.gate = p.epi == GEMM_EPI_GATE;
    prm.has_beta = beta != 0.0f || prm.gate;
    prm.has_bias = bias != nullptr;
    prm.relu = p.epi == GEMM_EPI_RELU || p.epi == GEMM_EPI_BIAS_RELU;
    prm.group_m = GROUP_M;
    prm.batch = prm.batch2 = 1;
    prm.stride_b = p.stride_b; prm.stride_bias = p.stride_bias; prm.stride_c = p.stride_c;
    prm.offs = offsets;
    prm.groups = (int)p.groups;
    prm.rows = (int)p.rows;
    prm.colsum = colsum;
    const GroupedEntry *k = p.fast && aligned(A, 16) && aligned(B, 16) ? p.fast : p.any;
    prm.tiles_m = (int)ceil_div(p.M, k->bm);
    prm.tiles_n = (int)ceil_div(p.N, k->bn);
    const unsigned grid = (unsigned)grid_of(p, *k, colsum != nullptr);
    if (grid == 0) return GEMM_STATUS_SUCCESS;
    return k->launch(prm, grid, static_cast<hipStream_t>(stream)) == hipSuccess ? GEMM_STATUS_SUCCESS
                                                                                : GEMM_STATUS_HIP_ERROR;
}

// Whether the kernel for few rows (16 rows per workgroup, K split over its waves) beats the tiles,
// which waste most of a tile but move more weights per workgroup: for a few rows per expert, and as
// long as its 16 x 64 workgroups (`few`) are about one round.  Measured (bf16, B not transposed, N 2048,
// K 4096; few rows -> best tile): 1 row per expert, 64 experts, 107 vs 146 us; 1 expert, 128 rows (272
// workgroups) 13 vs 30; 8 experts, 256 rows (640) 35 vs 44, 512 (1152) 49 vs 46, 1024 (2176) 81 vs 50;
// 64 experts, 512 rows (2048) 196 vs 193, 2048 (5120) 254 vs 200.
bool few_rows_pay(int64_t avg, double few) { return avg <= 6 || few <= 700; }

// Hands a finished plan out, with its description.
gemm_status_t finish_plan(gemm_grouped_plan_t *out, const gemm_grouped_plan &p, const char *what) {
    const GroupedEntry *k = p.fast ? p.fast : p.any;
    if (grid_of(p, *p.any, true) >= MAX_GRID || grid_of(p, *k, true) >= MAX_GRID) return GEMM_STATUS_NOT_SUPPORTED;
    gemm_grouped_plan *q = new (std::nothrow) gemm_grouped_plan(p);
    if (!q) return GEMM_STATUS_ALLOC_FAILED;
    snprintf(q->desc, sizeof q->desc, "grouped %s %s %s->%s tile %dx%d groups %lld grid %lld", what, k->name,
             type_name(p.ab), type_name(p.cd), k->bm, k->bn, (long long)p.groups,
             (long long)grid_of(p, *k, false));
    *out = q;
    return GEMM_STATUS_SUCCESS;
}

RowsFn rows16_table(int ab, int cd) {
    if (ab == GEMM_F16) return cd == GEMM_F16 ? tge::grouped_rows16_f16_f16 : tge::grouped_rows16_f16_f32;
    if (ab == GEMM_BF16) return cd == GEMM_BF16 ? tge::grouped_rows16_bf16_bf16 : tge::grouped_rows16_bf16_f32;
    return nullptr;
}

}  // namespace

extern "C" {

gemm_status_t gemm_grouped_plan_create(gemm_grouped_plan_t *out, const gemm_grouped_desc_t *d) {
    if (!out) return GEMM_STATUS_INVALID_VALUE;
    *out = nullptr;
    if (!d) return GEMM_STATUS_INVALID_VALUE;
    const int op_b = bits(d->op_b), ab = bits(d->ab_type), cd = bits(d->cd_type), epi = bits(d->epilogue),
              algo = bits(d->algo), tile = d->tile;
    if (!in(op_b, GEMM_OP_N, GEMM_OP_T) || !in(ab, GEMM_F32, GEMM_DF32) || !in(cd, GEMM_F32, GEMM_DF32) ||
        !in(epi, GEMM_EPI_NONE, GEMM_EPI_GATE))
        return GEMM_STATUS_INVALID_VALUE;
    switch (algo) {
    case GEMM_ALGO_AUTO: if (tile != 0) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_FAST: if (tile != 0 && tile != 256 && tile != 128 && tile != 64) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_FAST_STAGED: if (tile != 0 && tile != 128 && tile != 64) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_GENERAL: if (tile != 0 && tile != 128 && tile != 64) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_SKINNY:
        if (tile != 0 && tile != 64 && tile != (op_b == GEMM_OP_T ? 16 : 32)) return GEMM_STATUS_INVALID_VALUE;
        break;
    default: return GEMM_STATUS_INVALID_VALUE;
    }
    const gemm_status_t st = check_common(d->rows, d->N, d->K, d->groups, d->lda, d->ldb, d->ldc, ab, cd);
    if (st != GEMM_STATUS_SUCCESS) return st;
    const int64_t min_ldb = op_b == GEMM_OP_N ? d->N : d->K;
    if (d->lda < (d->K > 1 ? d->K : 1) || d->ldb < (min_ldb > 1 ? min_ldb : 1) ||
        d->ldc < (d->N > 1 ? d->N : 1) || d->stride_b < 0 || d->stride_bias < 0)
        return GEMM_STATUS_INVALID_VALUE;
    const int eab = elem_bytes(ab);
    // 32-bit offsets inside one expert's weights, 63-bit ones between them
    const int64_t b_rows = op_b == GEMM_OP_N ? d->K : d->N;
    const int64_t big = ((int64_t)1 << 62) / 8 / d->groups;
    if ((b_rows > 0 && (b_rows - 1) * d->ldb + min_ldb >= LIM31 / eab) || d->stride_b > big || d->stride_bias > big)
        return GEMM_STATUS_NOT_SUPPORTED;

    gemm_grouped_plan p = {};
    p.mode = tge::GROUP_ROWS;
    p.rows = d->rows; p.N = d->N; p.K = d->K; p.groups = d->groups;
    p.lda = d->lda; p.ldb = d->ldb; p.ldc = d->ldc; p.stride_b = d->stride_b; p.stride_bias = d->stride_bias;
    p.ab = ab; p.cd = cd; p.epi = epi;
    // Kernels: `any` runs whatever the pointers' alignment is, `fast` on aligned ones.
    const TableFn general = any_table(ab, cd);
    const bool t = op_b == GEMM_OP_T;
    const int64_t avg = ceil_div(d->rows, d->groups);                      // rows of an expert, on average
    const int64_t n = d->rows < d->groups ? d->rows : d->groups;           // experts with rows, at most
    const double tiles = ((double)d->rows / 128 + 0.5 * (double)n) * (double)ceil_div(d->N, 128);
    const double few = ((double)d->rows / 16 + 0.5 * (double)n) * (double)ceil_div(d->N, 64);
    const bool small = algo == GEMM_ALGO_GENERAL && tile ? tile == 64 : avg < 128 || d->N < 128;
    p.any = general(tge::GROUP_ROWS, op_b, small ? tge::CFG_64 : tge::CFG_128);
    const bool offsets_ok = d->lda * eab * 256 < LIM31;                    // 32-bit offsets within a tile's rows
    const bool staged_ok = eab == 2 && d->N >= 8 && d->K > 0 && offsets_ok;
    const bool rows16_ok = eab == 2 && d->K >= 8 && (t || d->N >= 8);
    // direct loads: whole 16-byte chunks
    const bool fast_ok = eab == 2 && d->K >= FAST_MIN_K && d->lda % 8 == 0 && d->ldb % 8 == 0 &&
                         d->stride_b % 8 == 0 && (t || (d->N % 8 == 0 && d->N > 0)) && offsets_ok;
    // 16 x 64 tiles where they give every CU a workgroup, else narrower ones.  Operands cold (in the
    // cache): B transposed 16 x 16 (4097 x 4097, one row, 24.7 -> 14.9 us (16.4 -> 12.0), 2048 x 4096 14.4 ->
    // 8.4 (9.8 -> 6.0); 200 rows over 8 experts, 1001 x 1001, 11.4 vs 13.8 (8.6 vs 11.5)), else 16 x 32 (2048 x
    // 4096, one row, 18.8 -> 17.1 us (10.9 -> 9.1), 4097 x 4097 23.9 -> 17.7 (16.6 -> 12.8); 200 rows over 8
    // experts, 1001 x 1001, 11.4 vs 12.3 (8.4 vs 9.4))
    const auto rows16 = [&]() {
        p.any = rows16_table(ab, cd)(op_b, 4);
        if (grid_of(p, *p.any, false) < 256) p.any = rows16_table(ab, cd)(op_b, t ? 1 : 2);
    };
    switch (algo) {
    case GEMM_ALGO_SKINNY:
        if (rows16_ok && tile) p.any = rows16_table(ab, cd)(op_b, tile / 16);
        else if (rows16_ok) rows16();
        break;
    case GEMM_ALGO_FAST:
        if (fast_ok) p.fast = fast_table(ab, cd)(tge::GROUP_ROWS, op_b, tile ? tile : 128, 0);
        break;
    case GEMM_ALGO_FAST_STAGED:
        if (staged_ok) p.any = fast_table(ab, cd)(tge::GROUP_ROWS, op_b, tile ? tile : 128, 1);
        break;
    case GEMM_ALGO_AUTO:
        if (rows16_ok && few_rows_pay(avg, few)) {
            rows16();
        } else {
            // 64-wide tiles where 128-wide ones are too few to fill the chip: 390 x 1968 x 2584 (56
            // of them) 33 -> 22 us, 1000 x 1000 x 1000 over 4 experts (78) 17 -> 12, 3000 x 776 x
            // 1000 over 7 (189) 18.2 -> 17.1; but 1000 x 4096 x 512 over 2 (281) 11.5 -> 13.4 and
            // 2100 x 1408 x 2048 over 32 (356) 46 -> 62
            if (fast_ok) {
                const int tl = wide_tiles_pay(d->rows, d->groups, n, avg, d->N, d->K) ? 256 : tiles < 200 ? 64 : 128;
                p.fast = fast_table(ab, cd)(tge::GROUP_ROWS, op_b, tl, 0);
            }
            // register-staged: 390 x 1968 x 2581 41 -> 23 us, 3001 x 777 x 1001 over 7 experts 28 -> 24, 700
            // x 4097 x 127 over 3 (231) 12 -> 10; but 20000 x 2049 x 4097 over 8 596 -> 984 (the
            // general kernel 1530, 87 for the second)
            if (staged_ok) p.any = fast_table(ab, cd)(tge::GROUP_ROWS, op_b, tiles < 400 ? 64 : 128, 1);
        }
        break;
    default: break;
    }
    char what[16];
    snprintf(what, sizeof what, "rows N%c", op_b == GEMM_OP_N ? 'N' : 'T');
    return finish_plan(out, p, what);
}

gemm_status_t gemm_grouped_grad_plan_create(gemm_grouped_plan_t *out, const gemm_grouped_grad_desc_t *d) {
    if (!out) return GEMM_STATUS_INVALID_VALUE;
    *out = nullptr;
    if (!d) return GEMM_STATUS_INVALID_VALUE;
    const int ab = bits(d->ab_type), cd = bits(d->cd_type), algo = bits(d->algo), tile = d->tile;
    if (!in(ab, GEMM_F32, GEMM_DF32) || !in(cd, GEMM_F32, GEMM_DF32)) return GEMM_STATUS_INVALID_VALUE;
    switch (algo) {
    case GEMM_ALGO_AUTO: if (tile != 0) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_FAST: if (tile != 0 && tile != 256 && tile != 128 && tile != 64) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_FAST_STAGED: if (tile != 0 && tile != 128 && tile != 64) return GEMM_STATUS_INVALID_VALUE; break;
    case GEMM_ALGO_GENERAL: if (tile != 0 && tile != 128 && tile != 64) return GEMM_STATUS_INVALID_VALUE; break;
    default: return GEMM_STATUS_INVALID_VALUE;
    }
    const gemm_status_t st = check_common(d->rows, d->N, d->M, d->groups, d->lda, d->ldb, d->ldc, ab, cd);
    if (st != GEMM_STATUS_SUCCESS) return st;
    if (d->rows > MAX_SUM_ROWS) return GEMM_STATUS_NOT_SUPPORTED;
    if (d->lda < (d->M > 1 ? d->M : 1) || d->ldb < (d->N > 1 ? d->N : 1) || d->ldc < (d->N > 1 ? d->N : 1))
        return GEMM_STATUS_INVALID_VALUE;
    const int64_t span = d->M > 0 && d->N > 0 ? (d->M - 1) * d->ldc + d->N : 0;
    if (d->stride_c < 0 || (d->groups > 1 && d->stride_c < span)) return GEMM_STATUS_INVALID_VALUE;
    if (d->stride_c > ((int64_t)1 << 62) / 8 / d->groups) return GEMM_STATUS_NOT_SUPPORTED;

    gemm_grouped_plan p = {};
    p.mode = tge::GROUP_K;
    p.rows = d->rows; p.M = d->M; p.N = d->N; p.groups = d->groups;
    p.lda = d->lda; p.ldb = d->ldb; p.ldc = d->ldc; p.stride_c = d->stride_c;
    p.ab = ab; p.cd = cd; p.epi = GEMM_EPI_NONE;
    const int eab = elem_bytes(ab);
    const bool small = algo == GEMM_ALGO_GENERAL && tile ? tile == 64 : d->M < 128 || d->N < 128;
    p.any = any_table(ab, cd)(tge::GROUP_K, 0, small ? tge::CFG_64 : tge::CFG_128);
    const bool staged_ok = eab == 2 && d->M >= 8 && d->N >= 8 && d->lda * eab * 256 < LIM31 &&
                           d->ldb * eab * 256 < LIM31;
    const int64_t avg = d->rows / d->groups;
    const int64_t tiles = d->groups * ceil_div(d->M, 128) * ceil_div(d->N, 128);
    // Register-staged: 64-wide tiles while the 128-wide ones do not fill the chip (3000 rows, 7 experts of
    // 1001 x 777, 26 -> 23 us, 300 rows, 16 of 333 x 1001, 11.1 -> 10.7; 16000 rows, 8 of 2049 x 2049,
    // 253 -> 381, 40 rows, 4 of 1955 x 7260, 84 -> 107; the general kernel 101 and 995 for the first
    // and third).
    if (staged_ok && algo != GEMM_ALGO_GENERAL)
        p.any = fast_table(ab, cd)(tge::GROUP_K, 0, algo == GEMM_ALGO_FAST_STAGED && tile ? tile : tiles < 400 ? 64 : 128, 1);
    const bool fast_ok = eab == 2 && d->M % 8 == 0 && d->N % 8 == 0 && d->M > 0 && d->N > 0 && d->lda % 8 == 0 &&
                         d->ldb % 8 == 0 && d->lda * eab * 256 < LIM31 && d->ldb * eab * 256 < LIM31;
    if (fast_ok && algo == GEMM_ALGO_FAST) p.fast = fast_table(ab, cd)(tge::GROUP_K, 0, tile ? tile : 128, 0);
    else if (fast_ok && algo == GEMM_ALGO_AUTO) {
        // The 256-wide tiles (one workgroup per CU, so that each tile's start and store are not
        // hidden) pay for long sums and nearly full rounds only.  Measured (bf16 -> fp32; 128 -> 256):
        // 32768 rows, one expert of 4096 x 4096 (256 wide tiles), 994 -> 772 us, 4 of them 986 -> 821,
        // 8192 rows, one of 8192 x 3328 (416) 439 -> 374; but one of 5120 x 4096 (320) 305 -> 344,
        // 16384 rows, 16 experts of 4096 x 2048, 356 -> 416, 32768 rows, 8 of 1024 x 1024 (128) 114 -> 138.
        const bool wide = avg >= 4096 && rounds_full(d->groups * ceil_div(d->M, 256) * ceil_div(d->N, 256));
        // 64-wide tiles where the 128-wide ones do not fill the chip or the sums are short: 1003
        // rows, 8 experts of 1024 x 704 (384 128-wide tiles), 12.1 -> 9.6 us, 2000 rows, 2 of 72 x
        // 3504, 17 -> 12, 40 rows, 4 of 1952 x 7264, 46 -> 42; 16000 rows, 8 of 2048 x 2048, 144 -> 192.
        p.fast = fast_table(ab, cd)(tge::GROUP_K, 0, wide ? 256 : tiles < 400 || avg < 64 ? 64 : 128, 0);
    }
    return finish_plan(out, p, "gradient TN");
}

// Checks shared by the two runs.
static gemm_status_t check_run(gemm_grouped_plan_t p, int mode, const void *A, const void *B, const void *C,
                               const void *D, const int32_t *offsets, float alpha, float beta, bool needs_c) {
    if (!p || p->mode != mode) return GEMM_STATUS_INVALID_VALUE;
    if (alpha != alpha || beta != beta) return GEMM_STATUS_INVALID_VALUE;   // NaN scalars
    const int eab = elem_bytes(p->ab), ecd = elem_bytes(p->cd);
    const bool has_d = mode == tge::GROUP_ROWS || p->M > 0;   // a gradient plan may have only sums
    if ((has_d && !D) || !offsets || !aligned(offsets, 4) || !aligned(D, ecd)) return GEMM_STATUS_INVALID_VALUE;
    const bool has_k = mode == tge::GROUP_ROWS ? p->K > 0 : p->rows > 0;
    if (has_k && (!A || !B || !aligned(A, eab) || !aligned(B, eab))) return GEMM_STATUS_INVALID_VALUE;
    if (needs_c && (!C || !aligned(C, ecd))) return GEMM_STATUS_INVALID_VALUE;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_grouped_run(gemm_grouped_plan_t p, const void *A, const void *B, const void *C, void *D,
                               const void *bias, const int32_t *offsets, float alpha, float beta, void *stream) {
    if (!p || p->mode != tge::GROUP_ROWS) return GEMM_STATUS_INVALID_VALUE;
    if (p->rows == 0 || p->N == 0) return GEMM_STATUS_SUCCESS;
    const bool gate = p->epi == GEMM_EPI_GATE;
    const gemm_status_t st = check_run(p, tge::GROUP_ROWS, A, B, C, D, offsets, alpha, beta, gate || beta != 0.0f);
    if (st != GEMM_STATUS_SUCCESS) return st;
    if (gate && beta != 0.0f) return GEMM_STATUS_INVALID_VALUE;
    const bool has_bias = p->epi == GEMM_EPI_BIAS || p->epi == GEMM_EPI_BIAS_RELU;
    if (has_bias && (!bias || !aligned(bias, 4))) return GEMM_STATUS_INVALID_VALUE;
    return launch(*p, A, B, C, D, has_bias ? bias : nullptr, nullptr, offsets, alpha, beta, stream);
}

gemm_status_t gemm_grouped_grad_run(gemm_grouped_plan_t p, const void *A, const void *B, const void *C, void *D,
                                    float *bias_grad, const int32_t *offsets, float alpha, float beta,
                                    void *stream) {
    if (!p || p->mode != tge::GROUP_K) return GEMM_STATUS_INVALID_VALUE;
    if (p->N == 0 || (p->M == 0 && !bias_grad)) return GEMM_STATUS_SUCCESS;
    const gemm_status_t st = check_run(p, tge::GROUP_K, A, B, C, D, offsets, alpha, beta, beta != 0.0f);
    if (st != GEMM_STATUS_SUCCESS) return st;
    if (!aligned(bias_grad, 4)) return GEMM_STATUS_INVALID_VALUE;
    return launch(*p, A, B, C, D, nullptr, bias_grad, offsets, alpha, beta, stream);
}

gemm_status_t gemm_grouped_plan_destroy(gemm_grouped_plan_t p) {
    delete p;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_grouped_plan_describe(gemm_grouped_plan_t p, char *buf, size_t len) {
    if (!p || !buf || len == 0) return GEMM_STATUS_INVALID_VALUE;
    snprintf(buf, len, "%s", p->desc);
    return GEMM_STATUS_SUCCESS;
}

}  // extern "C"
