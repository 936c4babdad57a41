// C ABI of a layer's products (bias, activation, residual; the gradient through the activation): plan
// creation and validation, kernel choice, launch.  Host code only; the kernels are the layer
// instances of gemm_kernels.hip and gemm_fast.hip, and layer_rows.hip.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/gemm.h"
#include "gemm_internal.h"
#include "host_common.h"

using namespace tge::host;
using tge::LayerEntry;
using tge::LayerParams;

struct gemm_layer_plan {
    int64_t rows, N, K, groups;
    int64_t lda, ldb, ldc, stride_b, stride_bias;
    int ab, cd, act;
    const LayerEntry *any;           // the kernel for any alignment: general, register-staged or for few rows
    const LayerEntry *fast;          // aligned pointers: the fast kernel with direct loads, else nullptr
    char desc[256];
};

namespace {

constexpr int64_t SLAB_BYTES = 128;        // of K: the fast kernel needs one

using TableFn = const LayerEntry *(*)(int, int);
using FastFn = const LayerEntry *(*)(int, int, int);

TableFn any_table(int ab, int cd) {
    if (ab == GEMM_F32 && cd == GEMM_F32) return tge::layer_any_f32_f32;
    if (ab == GEMM_F16 && cd == GEMM_F16) return tge::layer_any_f16_f16;
    if (ab == GEMM_F16 && cd == GEMM_F32) return tge::layer_any_f16_f32;
    if (ab == GEMM_BF16 && cd == GEMM_BF16) return tge::layer_any_bf16_bf16;
    if (ab == GEMM_BF16 && cd == GEMM_F32) return tge::layer_any_bf16_f32;
    return nullptr;
}

// The tables of the fast kernel and of the one for few rows.
FastFn fast_table(int ab, int cd) {
    if (ab == GEMM_F32) return tge::layer_fast_f32_f32;
    if (ab == GEMM_F16) return cd == GEMM_F16 ? tge::layer_fast_f16_f16 : tge::layer_fast_f16_f32;
    if (ab == GEMM_BF16) return cd == GEMM_BF16 ? tge::layer_fast_bf16_bf16 : tge::layer_fast_bf16_f32;
    return nullptr;
}
FastFn rows_table(int ab, int cd) {
    if (ab == GEMM_F32) return tge::layer_rows_f32_f32;
    if (ab == GEMM_F16) return cd == GEMM_F16 ? tge::layer_rows_f16_f16 : tge::layer_rows_f16_f32;
    if (ab == GEMM_BF16) return cd == GEMM_BF16 ? tge::layer_rows_bf16_bf16 : tge::layer_rows_bf16_f32;
    return nullptr;
}

// Workgroups of a launch, at most MAX_GRID; with one range and no offsets every one has a tile.
int64_t grid_of(const gemm_layer_plan &p, const LayerEntry &k) {
    const __int128 g = (__int128)row_tiles(p.rows, p.groups, k.bm) * ceil_div(p.N, k.bn);
    return g < MAX_GRID ? (int64_t)g : MAX_GRID;
}

// Whether D (and Z) are stored past the caches: as in the grouped plans, when rounds of tiles
// follow that read the operands again, except in rows off 64-byte lines after short sums.
bool stream_stores(const gemm_layer_plan &p, const LayerEntry &k, const void *D, int64_t grid, bool staged) {
    const int ecd = elem_bytes(p.cd);
    const bool apart = (((uintptr_t)D | (uintptr_t)(p.ldc * ecd)) & 63) != 0 && p.K <= (staged ? 32 : 512 / ecd);
    return !apart && grid > (k.bm == 256 ? 256 : 512);
}

// Whether the kernel for few rows reads the weights past the caches: where one workgroup reads each of them
// and all of them are half of the 256 MiB cache or more, so that they would not be found there
// anyway.  B transposed, 16 rows: 16384 x 4096 (128 MiB) in turn with three others 28.2 -> 23.3 us, alone
// 22.0 and 21.7; but 8192 x 4096 in turn 16.9 and 17.6, alone 13.3 and 17.1.  B not transposed (whose short
// pieces of rows lose their second halves): 4096 x 4096 in turn 12.5 -> 19.9.
bool read_once(const gemm_layer_plan &p, const LayerEntry &k) {
    return ceil_div(p.rows, p.groups) <= k.bm && (double)p.groups * p.K * p.N * elem_bytes(p.ab) >= (double)(128 << 20);
}

gemm_status_t launch(const gemm_layer_plan &p, LayerParams &prm, const void *A, const void *B, void *D,
                     const int32_t *offsets, float alpha, void *stream) {
    prm.A = A; prm.B = B; prm.D = D;
    prm.M = (int)p.rows; prm.N = (int)p.N; prm.K = (int)p.K;
    prm.lda = (int)p.lda; prm.ldb = (int)p.ldb; prm.ldc = (int)p.ldc;
    prm.alpha = alpha;
    prm.group_m = GROUP_M;
    prm.batch = prm.batch2 = 1;
    prm.stride_b = p.stride_b; prm.stride_bias = p.stride_bias;
    prm.offs = offsets;
    prm.groups = (int)p.groups;
    prm.rows = (int)p.rows;
    prm.act = p.act;
    const bool direct = p.fast && aligned(A, 16) && aligned(B, 16);
    const LayerEntry *k = direct ? p.fast : p.any;
    prm.tiles_m = (int)ceil_div(p.rows, k->bm);
    prm.tiles_n = (int)ceil_div(p.N, k->bn);
    const int64_t grid = grid_of(p, *k);
    prm.once = read_once(p, *k);
    prm.stream = stream_stores(p, *k, D, grid, !direct);
    return k->launch(prm, (unsigned)grid, static_cast<hipStream_t>(stream)) == hipSuccess ? GEMM_STATUS_SUCCESS
                                                                                          : GEMM_STATUS_HIP_ERROR;
}

// What both runs check; the plan is not empty.
gemm_status_t check_run(const gemm_layer_plan &p, const void *A, const void *B, const void *D,
                        const int32_t *offsets, float alpha) {
    if (alpha != alpha) return GEMM_STATUS_INVALID_VALUE;   // NaN
    const int eab = elem_bytes(p.ab);
    if (!D || !aligned(D, elem_bytes(p.cd))) return GEMM_STATUS_INVALID_VALUE;
    if (p.K > 0 && (!A || !B || !aligned(A, eab) || !aligned(B, eab))) return GEMM_STATUS_INVALID_VALUE;
    if (offsets ? !aligned(offsets, 4) : p.groups > 1) return GEMM_STATUS_INVALID_VALUE;
    return GEMM_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

gemm_status_t gemm_layer_plan_create(gemm_layer_plan_t *out, const gemm_layer_desc_t *d) {
    if (!out) return GEMM_STATUS_INVALID_VALUE;
    *out = nullptr;
    if (!d) return GEMM_STATUS_INVALID_VALUE;
    const int op_b = bits(d->op_b), ab = bits(d->ab_type), cd = bits(d->cd_type), act = bits(d->act),
              algo = bits(d->algo), tile = d->tile;
    if (!in(op_b, GEMM_OP_N, GEMM_OP_T) || !in(ab, GEMM_F32, GEMM_DF32) || !in(cd, GEMM_F32, GEMM_DF32) ||
        !in(act, GEMM_ACT_NONE, GEMM_ACT_SILU))
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
    if (d->rows < 0 || d->N < 0 || d->K < 0 || d->groups < 1) return GEMM_STATUS_INVALID_VALUE;
    if (d->rows >= LIM31 || d->N >= LIM31 || d->K >= LIM31 || d->lda >= LIM31 || d->ldb >= LIM31 ||
        d->ldc >= LIM31 || d->groups >= MAX_GROUPS || !any_table(ab, cd))
        return GEMM_STATUS_NOT_SUPPORTED;
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

    gemm_layer_plan p = {};
    p.rows = d->rows; p.N = d->N; p.K = d->K; p.groups = d->groups;
    p.lda = d->lda; p.ldb = d->ldb; p.ldc = d->ldc; p.stride_b = d->stride_b; p.stride_bias = d->stride_bias;
    p.ab = ab; p.cd = cd; p.act = act;
    // Kernels: `any` runs whatever the pointers' alignment is, `fast` on aligned ones.  The rules for the
    // tiles are those of the grouped plans, where they are measured.
    const bool t = op_b == GEMM_OP_T;
    const int64_t avg = ceil_div(d->rows, d->groups);                      // rows of an expert, on average
    const int64_t n = d->rows < d->groups ? d->rows : d->groups;           // experts with rows, at most
    const double ragged = d->groups > 1 ? 0.5 * (double)n : 0.0;           // half a tile at each range's end
    const double tiles = ((double)d->rows / 128 + ragged) * (double)ceil_div(d->N, 128);
    const double few = ((double)d->rows / 16 + ragged) * (double)ceil_div(d->N, 64);
    const bool small = algo == GEMM_ALGO_GENERAL && tile ? tile == 64 : avg < 128 || d->N < 128;
    p.any = any_table(ab, cd)(op_b, small ? tge::CFG_64 : tge::CFG_128);
    const bool offsets_ok = d->lda * eab * 256 < LIM31;                    // 32-bit offsets within a tile's rows
    const int64_t ve = 16 / eab;
    const bool staged_ok = d->N >= ve && d->K > 0 && offsets_ok;
    const bool rows_ok = d->K >= ve && (t || d->N >= ve) && d->lda * eab * 64 < LIM31;
    // direct loads: whole 16-byte chunks
    const bool fast_ok = d->K >= SLAB_BYTES / eab && d->lda % ve == 0 && d->ldb % ve == 0 &&
                         d->stride_b % ve == 0 && (t || (d->N % ve == 0 && d->N > 0)) && offsets_ok;
    // Rounds of 256 workgroups that the tiles make (about, with ranges).
    const auto rounds = [&](int bm, int bn) {
        const double per = (double)avg / bm + 0.5;                             // row tiles of an expert
        const double down = d->groups == 1 ? (double)ceil_div(d->rows, bm) : (double)n * (per > 1 ? per : 1);
        const double grid = down * (double)ceil_div(d->N, bn);
        return grid <= 256 ? 1.0 : d->groups == 1 ? (double)ceil_div((int64_t)grid, 256) : grid / 256;
    };
    // The kernel for few rows.  Its workgroups load some 50 GB/s each, so a shape costs what one of them
    // loads, 16 (rt + cg) rows of K, times the rounds of 256; and, in fp32, part of its matrix instructions:
    // 16 x 4096 x 4096 9.6 us in 16 columns (256 workgroups), 12.8 in 64 (64 of them); 64 x 4096 x 16384 47 in
    // 64 x 16, 76 in 64 x 64; 64 x 6144 x 4096 23.6 and 20.1; fp32, 64 x 1024 x 8192 53 in 64 x 16, 19 in 16 x 16.
    const auto rows_kernel = [&](int cg) {
        double least = 0;
        for (const int r : {1, 2, 4})
            for (const int c : {4, t ? 1 : 2}) {
                const double cost = rounds(16 * r, 16 * c) * (r + c + (eab == 4 ? 0.4 * r * c : 0.0));
                if ((cg == 0 || c == cg) && (least == 0 || cost < least)) {
                    least = cost;
                    p.any = rows_table(ab, cd)(op_b, r, c);
                }
            }
        return least;
    };
    // Whether that kernel beats the tiles.  One matrix, gelu: up to 64 rows (64 x 65536 x 4096 121 -> 110
    // us), and while its workgroups are one round, or two of long sums (256 x 4096 x 4096 32 -> 21, 384 x
    // 4096 x 16384 175 -> 124, but 512 x 4096 x 4096 32 vs 36, 192 x 16384 x 4096 58 vs 66).  Experts' ranges
    // are ragged, and read weights of their own, by ever more waves (us, tiles -> few rows; B transposed): 8
    // rows each, 128 of 1536 x 2048 147 -> 138, 64 of 2048 x 4096 174 -> 169; 16 and 24 rows, 64 of 768 x 2048
    // 52 -> 47 and 53 -> 49, 8 of 2048 x 4096 46 -> 33 and 46 -> 38, but 64 of 2048 x 4096 174 vs 200 and 180 vs
    // 204; 64 rows, 16 of 1024 x 2048 21 vs 25.  Not transposed: 2 rows, 64 of 2048 x 4096 165 -> 157, 8 and
    // 24 rows, 8 of them, 39 -> 26 and 40 -> 38, but 8 rows, 64 of 768 x 2048 38 vs 50.
    const auto few_rows = [&]() {
        if (d->groups == 1) {
            const int64_t wide = ceil_div(d->rows, 64) * ceil_div(d->N, 64);
            return d->rows <= 64 || wide <= 256 || (wide <= 512 && d->K >= 8192);
        }
        return t ? avg <= 8 || (avg <= 32 && few <= 1600) : avg <= 4 || few <= 700;
    };
    switch (algo) {
    case GEMM_ALGO_SKINNY:
        if (rows_ok) rows_kernel(tile / 16);
        break;
    case GEMM_ALGO_FAST:
        if (fast_ok) p.fast = fast_table(ab, cd)(op_b, tile ? tile : 128, 0);
        break;
    case GEMM_ALGO_FAST_STAGED:
        if (staged_ok) p.any = fast_table(ab, cd)(op_b, tile ? tile : 128, 1);
        break;
    case GEMM_ALGO_AUTO:
        if (eab == 4) {
            // The least of what a round costs, in the kernel for few rows' unit (1.5 us per 1000 of K): bound by
            // the matrix instructions, of 64 x 64 tiles 10.5, of 128 x 128 ones 37 (a start that nothing hides in
            // short sums), register-staged 15 and 45.  us of 64 x 64, 128 x 128 tiles and the kernel for few rows,
            // K 4096, N 4096: 128 rows 67, 233, 50; 256 rows 72, 234, 88; 512 rows 132, 233, 170; 2048 rows 490, 464,
            // 628; register-staged 512 rows 177, 287; 2048 rows 642, 541; N 1024, 4096 rows, K 256 24, 28, 38
            const double k = (double)(d->K > 1 ? d->K : 1), start = 2000.0 / k, r64 = rounds(64, 64), r128 = rounds(128, 128);
            const double rows_cost = rows_ok ? rows_kernel(0) * (1.0 + 100.0 / k) : INFINITY;
            const double fast64 = 10.5 * r64, fast128 = (37.0 + start) * r128, staged64 = 15.0 * r64, staged128 = (45.0 + start) * r128;
            if (staged_ok && fmin(staged64, staged128) < rows_cost) p.any = fast_table(ab, cd)(op_b, staged64 <= staged128 ? 64 : 128, 1);
            if (fast_ok && fmin(fast64, fast128) < rows_cost) p.fast = fast_table(ab, cd)(op_b, fast64 <= fast128 ? 64 : 128, 0);
        } else if (rows_ok && few_rows()) {
            rows_kernel(0);
        } else {
            if (fast_ok) {
                // 64-wide tiles also for short ranges of a transposed B: 24 rows, 64 experts of 2048 x 4096 184
                // -> 180 us, 16 rows, 128 of 1536 x 2048 159 -> 150; 32 rows 187 vs 219
                const int tl = wide_tiles_pay(d->rows, d->groups, n, avg, d->N, d->K) ? 256
                               : tiles < 200 || (t && avg <= 24) ? 64 : 128;
                p.fast = fast_table(ab, cd)(op_b, tl, 0);
            }
            if (staged_ok) p.any = fast_table(ab, cd)(op_b, tiles < 400 ? 64 : 128, 1);
        }
        break;
    default: break;
    }
    const LayerEntry *k = p.fast ? p.fast : p.any;
    if (grid_of(p, *p.any) >= MAX_GRID || grid_of(p, *k) >= MAX_GRID) return GEMM_STATUS_NOT_SUPPORTED;
    gemm_layer_plan *q = new (std::nothrow) gemm_layer_plan(p);
    if (!q) return GEMM_STATUS_ALLOC_FAILED;
    static const char *const names[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};
    snprintf(q->desc, sizeof q->desc, "layer N%c %s %s %s->%s tile %dx%d groups %lld grid %lld", t ? 'T' : 'N',
             names[act], k->name, type_name(ab), type_name(cd), k->bm, k->bn, (long long)p.groups,
             (long long)grid_of(p, *k));
    *out = q;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_layer_run(gemm_layer_plan_t p, const void *A, const void *B, const void *C, void *D, void *Z,
                             const void *bias, const int32_t *offsets, float alpha, float beta, void *stream) {
    if (!p) return GEMM_STATUS_INVALID_VALUE;
    if (p->rows == 0 || p->N == 0) return GEMM_STATUS_SUCCESS;
    const gemm_status_t st = check_run(*p, A, B, D, offsets, alpha);
    if (st != GEMM_STATUS_SUCCESS) return st;
    const int ecd = elem_bytes(p->cd);
    if (beta != beta || (beta != 0.0f && (!C || !aligned(C, ecd))) || (bias && !aligned(bias, 4)))
        return GEMM_STATUS_INVALID_VALUE;
    if (Z && (!aligned(Z, ecd) || Z == D || (beta != 0.0f && Z == C))) return GEMM_STATUS_INVALID_VALUE;
    LayerParams prm = {};
    prm.C = C; prm.Z = Z; prm.bias = bias;
    prm.beta = beta;
    prm.has_beta = beta != 0.0f;
    prm.has_bias = bias != nullptr;
    return launch(*p, prm, A, B, D, offsets, alpha, stream);
}

gemm_status_t gemm_layer_grad_run(gemm_layer_plan_t p, const void *A, const void *B, const void *Z, void *D,
                                  const int32_t *offsets, float alpha, void *stream) {
    if (!p) return GEMM_STATUS_INVALID_VALUE;
    if (p->rows == 0 || p->N == 0) return GEMM_STATUS_SUCCESS;
    const gemm_status_t st = check_run(*p, A, B, D, offsets, alpha);
    if (st != GEMM_STATUS_SUCCESS) return st;
    // without an activation the slope is 1 and Z is not read
    const bool reads = p->act != tge::ACT_NONE;
    if (reads && (!Z || !aligned(Z, elem_bytes(p->cd)))) return GEMM_STATUS_INVALID_VALUE;
    LayerParams prm = {};
    prm.Z = reads ? const_cast<void *>(Z) : nullptr;
    prm.grad = reads;
    return launch(*p, prm, A, B, D, offsets, alpha, stream);
}

gemm_status_t gemm_layer_plan_destroy(gemm_layer_plan_t p) {
    delete p;
    return GEMM_STATUS_SUCCESS;
}

gemm_status_t gemm_layer_plan_describe(gemm_layer_plan_t p, char *buf, size_t len) {
    if (!p || !buf || len == 0) return GEMM_STATUS_INVALID_VALUE;
    snprintf(buf, len, "%s", p->desc);
    return GEMM_STATUS_SUCCESS;
}

}  // extern "C"
