// Internal interface between the host plan/run code and the device kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tge {

// Everything a kernel needs for one launch; passed by value as the kernel argument.
struct GemmParams {
    const void *A, *B, *C;
    void *D;
    const void *bias;
    int M, N, K;
    int lda, ldb, ldc;       // elements of each matrix's own type
    float alpha, beta;
    int has_beta, has_bias, relu;
    int tiles_m, tiles_n;    // output tiles along M and N (of one product)
    int group_m;             // tile rows per raster group
    // strided batch: the launch computes `batch` independent products; product b reads and
    // writes the operands moved by b * stride (in elements of each operand's own type; C and D
    // share stride_c; a zero stride shares that operand between products).  With a second batch
    // mode (batch2 > 1) `batch` counts all products and product b = b1 * batch2 + b2 is moved by
    // b1 * stride + b2 * stride2
    int batch;
    int64_t stride_a, stride_b, stride_c, stride_bias;
    int batch2;
    int64_t stride2_a, stride2_b, stride2_c, stride2_bias;
    // load transforms (1: zero every element whose sign bit is set) on op(A), op(B) and C
    int xform_a, xform_b, xform_c;
    // split-K workspace of the skinny kernel (partial sums of every k split); unused elsewhere
    float *ws;
};

using LaunchFn = hipError_t (*)(const GemmParams &, unsigned grid, hipStream_t);

// One launch of products grouped by expert: the operands' rows are cut into `groups` ranges,
// range e = [offs[e], offs[e+1]) with offs in device memory (groups + 1 values).
//   GROUP_ROWS  the ranges cut the rows of A, C and D; range e is multiplied by B + e * stride_b
//               (bias + e * stride_bias); M is set per workgroup
//   GROUP_K     the ranges cut the product's K, the stored rows of both operands (A stored
//               transposed, B not): product e sums over range e into D + e * stride_c; K is set
//               per workgroup
// A range is clamped to [0, rows], so that no offset makes a kernel leave the operands.
//   GROUP_LAYER as GROUP_ROWS, with a layer's epilogue (LayerParams); without offsets all rows are
//               one range
enum GroupMode { GROUP_NONE = 0, GROUP_ROWS = 1, GROUP_K = 2, GROUP_LAYER = 3 };
constexpr int COLSUM_COLS = 64;   // columns of a workgroup that sums B (gradient plans)
struct GroupedParams : GemmParams {
    const int32_t *offs;
    int groups, rows;
    int gate;                // GROUP_ROWS: D = C > 0 ? alpha * product : 0 (has_beta set: C is read)
    float *colsum;           // GROUP_K: column sums of B per range, groups x N (nullptr: none)
};
using GroupedLaunchFn = hipError_t (*)(const GroupedParams &, unsigned grid, hipStream_t);
struct GroupedEntry {
    GroupedLaunchFn launch;
    int bm, bn;              // workgroup tile
    const char *name;
};

// One launch of a layer's products (GROUP_LAYER).  Forward: z = alpha * product + bias, D = act(z) +
// beta * C (C read where has_beta is set), z written to Z where it is not nullptr.  grad: D =
// act'(Z) * alpha * product, Z read.  Z is laid out like D.
enum ActKind { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };
struct LayerParams : GroupedParams {
    void *Z;
    int act, grad;
    int stream;              // stores past the caches
    int once;                // few rows: weights past them too
};
using LayerLaunchFn = hipError_t (*)(const LayerParams &, unsigned grid, hipStream_t);
struct LayerEntry {
    LayerLaunchFn launch;
    int bm, bn;              // workgroup tile
    const char *name;
};

// One compiled kernel variant and its tile shape.
struct KernelEntry {
    LaunchFn launch;
    int bm, bn, bk;          // workgroup tile (bk in elements)
    int waves_m, waves_n;    // wave grid inside the workgroup
    const char *name;
};

// Tile configurations, largest first.
enum TileCfg { CFG_256 = 0, CFG_128 = 1, CFG_64 = 2, CFG_COUNT = 3 };

// Per type-pair lookup, defined by the kernel translation units (one per pair).
// op_a/op_b: 0 = N, 1 = T.  Returns nullptr for an unknown combination.
const KernelEntry *kernels_f32_f32(int op_a, int op_b, int cfg);
const KernelEntry *kernels_f16_f16(int op_a, int op_b, int cfg);
const KernelEntry *kernels_f16_f32(int op_a, int op_b, int cfg);
const KernelEntry *kernels_bf16_bf16(int op_a, int op_b, int cfg);
const KernelEntry *kernels_bf16_f32(int op_a, int op_b, int cfg);
const KernelEntry *kernels_i8_i32(int op_a, int op_b, int cfg);

// Products with a diagonal operand (gemm_diag.hip), streamed: dg bit 0 = A diagonal, bit 1 =
// B diagonal; the op of the dense operand picks the kernel.  No alignment preconditions.
const KernelEntry *diag_f32_f32(int op_a, int op_b, int dg);
const KernelEntry *diag_f16_f16(int op_a, int op_b, int dg);
const KernelEntry *diag_f16_f32(int op_a, int op_b, int dg);
const KernelEntry *diag_bf16_bf16(int op_a, int op_b, int dg);
const KernelEntry *diag_bf16_f32(int op_a, int op_b, int dg);
const KernelEntry *diag_i8_i32(int op_a, int op_b, int dg);

// Fast 256x256 path for 16- and 8-bit inputs (gemm_fast.hip); K >= one slab (64 elements, 128
// for int8).  rs = 0: direct-to-LDS loads; needs 16-byte aligned A/B pointers, leading dimensions
// and batch strides, and M (when A is stored transposed) and N (when B is not) multiples of
// 16 / element size.  rs = 1: register-staged loads, no alignment or extent preconditions.
const KernelEntry *fast_f16_f16(int op_a, int op_b, int rs);
const KernelEntry *fast_f16_f32(int op_a, int op_b, int rs);
const KernelEntry *fast_bf16_bf16(int op_a, int op_b, int rs);
const KernelEntry *fast_bf16_f32(int op_a, int op_b, int rs);
const KernelEntry *fast_i8_i32(int op_a, int op_b, int rs);
// The same kernel with 128x128 tiles (4 waves of 64x64, two workgroups per CU) for mid-size
// products: direct loads only (the same alignment preconditions), no load transforms on
// op(A)/op(B).
const KernelEntry *fast128_f16_f16(int op_a, int op_b);
const KernelEntry *fast128_f16_f32(int op_a, int op_b);
const KernelEntry *fast128_bf16_bf16(int op_a, int op_b);
const KernelEntry *fast128_bf16_f32(int op_a, int op_b);
const KernelEntry *fast128_i8_i32(int op_a, int op_b);

// Byte-exact copy of an operand into rows that are 16-byte aligned and zero-padded to whole
// 16-byte chunks (gemm_repack.hip), for operands the direct loads cannot take: row r < rows of
// product b goes from src + b * src_stride + r * src_pitch (row_bytes bytes) to
// dst + b * dst_stride + r * dst_pitch, rows rows .. rows_out - 1 are written as zeros (all in
// bytes; dst, dst_pitch and dst_stride multiples of 16, dst_pitch >= row_bytes, rows_out >=
// rows).  repack_launch copies a and b (rows_out == 0: no job) in one launch; the caller keeps
// the total of repack_blocks below 2^31.
// With xf_elem = 1 or 2 the copy also applies the load transform GEMM_TRANSFORM_RELU to
// elements of that many bytes (every element whose sign bit is set becomes +0).
// tr_elem = 1 or 2 makes the copy transposing, for elements of that many bytes: the source's
// `rows` rows (k) of row_bytes / tr_elem elements (m) become row_bytes / tr_elem destination
// rows of rows_out elements each (k; zero for k >= rows), row m at dst + b * dst_stride +
// m * dst_pitch; rows_out * tr_elem a multiple of 128, src_pitch a multiple of tr_elem.
struct RepackJob {
    const uint8_t *src;
    uint8_t *dst;
    int64_t rows, rows_out, row_bytes, src_pitch, dst_pitch, src_stride, dst_stride, batch;
    int xf_elem;
    int tr_elem;
};
int64_t repack_blocks(const RepackJob &j);
hipError_t repack_launch(const RepackJob &a, const RepackJob &b, hipStream_t stream);

// Type-converting copy (gemm_repack.hip): an operand stored as fp32 (src_type
// CONVERT_FROM_F32, rounded to nearest even) or int8 (CONVERT_FROM_I8, exact) becomes fp16 (or
// bf16 with to_bf16) rows.  Row r < rows of product b holds `elems` source elements at
// src + b * src_stride + r * src_pitch (bytes, any alignment); it is written to
// dst + b * dst_stride + r * dst_pitch (dst, dst_pitch and dst_stride multiples of 16;
// dst_pitch >= 2 * elems), zero past the row's elements.  convert_launch converts a and b
// (rows == 0: no job) in one launch; the caller keeps the total of convert_blocks below 2^31.
enum ConvertSrc { CONVERT_FROM_F32 = 0, CONVERT_FROM_I8 = 1 };
struct ConvertJob {
    const uint8_t *src;
    uint8_t *dst;
    int64_t rows, elems, src_pitch, dst_pitch, src_stride, dst_stride, batch;
    int src_type, to_bf16;
};
int64_t convert_blocks(const ConvertJob &j);
hipError_t convert_launch(const ConvertJob &a, const ConvertJob &b, hipStream_t stream);

// Complex / dual operands with fp16 parts rewritten as real fp16 matrices for the real kernels
// (gemm_repack.hip).  Source row r of product b holds `numbers` numbers (4 bytes each: real
// part low, other part high) at src + b * src_stride + r * src_pitch; it becomes destination
// rows 2r and 2r+1 at dst + b * dst_stride + (2r + h) * dst_pitch (bytes; dst_pitch a multiple
// of 16, zero-padded past the data):
//   PAIR_PARTS    row 2r: the real parts, row 2r+1: the other parts (numbers fp16 values each)
//   PAIR_BLOCK_N  row 2r: (re, im) pairs as stored, row 2r+1: (-im, re) pairs, dual (0, re)
//   PAIR_BLOCK_T  row 2r: (re, -im) pairs, dual (re, 0), row 2r+1: (im, re) pairs
// A complex product is then a real one: with op(A) read as M x 2K reals (parts interleaved
// along K) and each number b of op(B) replaced by the 2 x 2 block [re im; -im re] (dual:
// [re im; 0 re]), D read as M x 2N reals is op(A) times the 2K x 2N block matrix.
enum PairMode { PAIR_PARTS = 0, PAIR_BLOCK_N = 1, PAIR_BLOCK_T = 2 };
struct PairJob {
    const uint8_t *src;
    uint8_t *dst;
    int64_t rows, numbers, src_pitch, dst_pitch, src_stride, dst_stride, batch;
    int mode, dual;
};
int64_t pair_blocks(const PairJob &j);
hipError_t pair_launch(const PairJob &a, const PairJob &b, hipStream_t stream);

// Complex and dual GEMM (gemm_complex.hip): fp16 parts, fp32 accumulation, 128x128 tile.
const KernelEntry *complex_cf16_cf32(int op_a, int op_b);
const KernelEntry *complex_cf16_cf16(int op_a, int op_b);
const KernelEntry *complex_df16_df32(int op_a, int op_b);
const KernelEntry *complex_df16_df16(int op_a, int op_b);

// Memory-bound path for M <= 64 (gemm_skinny.hip); mt = ceil(M / 16).  Preconditions: 16-bit
// inputs, or int8 inputs with B transposed (op_b == T); op_a == N, K a whole number of 64-byte
// chunks (K % 32 == 0 for 16-bit inputs, K % 64 == 0 for int8), 16-byte aligned A/B pointers and
// leading dimensions, N % 8 == 0 when B is not transposed.  One workgroup per bn (64) columns and k split: the
// launch sets tiles_m = S (k splits), tiles_n = ceil(N / bn), grid = S * tiles_n * batch, and
// with S > 1 passes the workspace ws (batch * S * M * N floats); the entry then enqueues a
// second, finishing kernel.  narrow = 1 (B transposed only): 16 columns per workgroup, S = 1.
const KernelEntry *skinny_f16_f16(int op_b, int mt, int narrow);
const KernelEntry *skinny_f16_f32(int op_b, int mt, int narrow);
const KernelEntry *skinny_bf16_bf16(int op_b, int mt, int narrow);
const KernelEntry *skinny_bf16_f32(int op_b, int mt, int narrow);
const KernelEntry *skinny_i8_i32(int op_b, int mt, int narrow);   // op_b == T only; S > 1: one product

// The finishing step alone: D = epilogue(sum over the p.tiles_m splits of ws, in split order),
// ws laid out [product][split][M][N] floats; p otherwise as for the product (C, bias, ldc,
// alpha, beta, ReLU, the C transform).  Used by the fast kernel's K split too.
hipError_t finish_f16_f16(const GemmParams &p, hipStream_t s);
hipError_t finish_f16_f32(const GemmParams &p, hipStream_t s);
hipError_t finish_bf16_bf16(const GemmParams &p, hipStream_t s);
hipError_t finish_bf16_f32(const GemmParams &p, hipStream_t s);
// int8 -> int32 (gemm_repack.hip): int32 partial sums in ws, one product (batch 1)
hipError_t finish_i8_i32(const GemmParams &p, hipStream_t s);

// Grouped products (the same kernels with the group selection compiled in).  mode: GroupMode;
// op_b: 0 = N, 1 = T (GROUP_K: 0).  Preconditions as for the kernels above, for every range:
//   any    the general kernel, tile CFG_128 or CFG_64: none
//   fast   tile 256, 128 or 64, direct loads: 16-byte aligned pointers, leading dimensions and strides;
//          GROUP_ROWS: K >= 64, N % 8 == 0 when op_b is N; GROUP_K: M % 8 == 0 and N % 8 == 0.
//          rs = 1 (tile 128 or 64): register-staged loads; at least 8 elements (one chunk) along M and N,
//          nothing else
//   rows16 GROUP_ROWS, 16 rows and 16 * cg columns per workgroup (cg 4, or 1 when op_b is T, 2
//          when it is N): K >= 8, N >= 8 when op_b is N
const GroupedEntry *grouped_any_f32_f32(int mode, int op_b, int cfg);
const GroupedEntry *grouped_any_f16_f16(int mode, int op_b, int cfg);
const GroupedEntry *grouped_any_f16_f32(int mode, int op_b, int cfg);
const GroupedEntry *grouped_any_bf16_bf16(int mode, int op_b, int cfg);
const GroupedEntry *grouped_any_bf16_f32(int mode, int op_b, int cfg);
const GroupedEntry *grouped_fast_f16_f16(int mode, int op_b, int tile, int rs);
const GroupedEntry *grouped_fast_f16_f32(int mode, int op_b, int tile, int rs);
const GroupedEntry *grouped_fast_bf16_bf16(int mode, int op_b, int tile, int rs);
const GroupedEntry *grouped_fast_bf16_f32(int mode, int op_b, int tile, int rs);
const GroupedEntry *grouped_rows16_f16_f16(int op_b, int cg);
const GroupedEntry *grouped_rows16_f16_f32(int op_b, int cg);
const GroupedEntry *grouped_rows16_bf16_bf16(int op_b, int cg);
const GroupedEntry *grouped_rows16_bf16_f32(int op_b, int cg);

// A layer's products: any and fast are the kernels of GROUP_ROWS, under the same preconditions.
const LayerEntry *layer_any_f32_f32(int op_b, int cfg);
const LayerEntry *layer_any_f16_f16(int op_b, int cfg);
const LayerEntry *layer_any_f16_f32(int op_b, int cfg);
const LayerEntry *layer_any_bf16_bf16(int op_b, int cfg);
const LayerEntry *layer_any_bf16_f32(int op_b, int cfg);
const LayerEntry *layer_fast_f32_f32(int op_b, int tile, int rs);
const LayerEntry *layer_fast_f16_f16(int op_b, int tile, int rs);
const LayerEntry *layer_fast_f16_f32(int op_b, int tile, int rs);
const LayerEntry *layer_fast_bf16_bf16(int op_b, int tile, int rs);
const LayerEntry *layer_fast_bf16_f32(int op_b, int tile, int rs);
//   rows   16 * rt rows and 16 * cg columns per workgroup (rt 1, 2 or 4; cg 4, or 1 when op_b is T, 2
//          when it is N): K of a 16-byte chunk, N too when op_b is N; 64 rows of A within 2^31 bytes
const LayerEntry *layer_rows_f32_f32(int op_b, int rt, int cg);
const LayerEntry *layer_rows_f16_f16(int op_b, int rt, int cg);
const LayerEntry *layer_rows_f16_f32(int op_b, int rt, int cg);
const LayerEntry *layer_rows_bf16_bf16(int op_b, int rt, int cg);
const LayerEntry *layer_rows_bf16_f32(int op_b, int rt, int cg);

// Products with 4-bit weights (gemm_quant.hip): W_e[n][k] = scale * (code - zero), codes packed
// two per byte along k (low half: even k), one scale (of A's type) and zero point (uint8; nullptr:
// 8) per `block` consecutive k.  offs == nullptr: one weight matrix for all rows.
struct QuantParams : GroupedParams {
    const uint8_t *Q;        // codes: expert e, row n at Q + e * stride_q + n * ldq (bytes)
    const void *scales;      // expert e, row n, block b at e * stride_s + n * lds + b (elements)
    const uint8_t *zeros;    // laid out like the scales
    int64_t stride_q, stride_s;
    int ldq, lds, block;
    uint64_t block_rcp;      // ceil(2^32 / (block / 128)) for blocks of 128 and more
};
using QuantLaunchFn = hipError_t (*)(const QuantParams &, unsigned grid, hipStream_t);
struct QuantEntry {
    QuantLaunchFn launch;
    int bm, bn;              // workgroup tile
    const char *name;
};
// block: 32, 64, or 128 for every multiple of 128 (K a multiple of the block).  No alignment
// preconditions beyond the elements' own.
//   rows:  16 x 16 * cg tiles (cg 1 or 4), K split over the waves of a workgroup
//   tile:  128 x 128 tiles
const QuantEntry *quant_rows_f16_f16(int block, int cg);
const QuantEntry *quant_rows_f16_f32(int block, int cg);
const QuantEntry *quant_rows_bf16_bf16(int block, int cg);
const QuantEntry *quant_rows_bf16_f32(int block, int cg);
const QuantEntry *quant_tile_f16_f16(int block);
const QuantEntry *quant_tile_f16_f32(int block);
const QuantEntry *quant_tile_bf16_bf16(int block);
const QuantEntry *quant_tile_bf16_f32(int block);

// Layer norm (layer_norm.hip).  A row belongs to a team of `waves` waves, whose lanes hold 16-byte
// chunks lane, lane + 64 * waves, ... (`chunks` of them) of it; N elements fill at most the team's
// chunks.  Workgroups have `teams` teams and take rows blockIdx * teams + team, then every
// grid * teams-th; a row that needs fewer lanes than a wave has `lanes` of them, and 64 / lanes rows stand side by
// side in a team.  Pointers need their elements' alignment only.
struct NormParams {
    const void *X;           // rows x N, ldx
    const float *weight, *bias;      // nullptr: 1 and 0
    void *Y;                 // rows x N, ldy (gradient: dY, read)
    float *mean, *rstd;      // one per row; forward: nullptr leaves them out
    const void *C;           // gradient: dX = ... + beta * C (read where has_beta is set), ldx
    void *dX;                // ldx
    float *part;             // gradient: grid x 2 x N partial sums (weight's, bias's); nullptr: none
    int rows, N, ldx, ldy;
    float eps, rn;           // 1 / N
    float beta;
    int has_beta;
};
struct NormShape {
    int waves, chunks, teams, lanes;
};
// Teams of a workgroup, which so has 4 waves, or 8 in the gradient, unless one row needs more.
constexpr int norm_teams(int waves, bool grad) { return waves < (grad ? 8 : 4) ? (grad ? 8 : 4) / waves : 1; }
// The team of a row of `pieces` (1 to 4096) 16-byte chunks: one per lane, or two, in as few waves as hold it;
// more than two (of 16 waves) for the longest rows only, as they cost the registers that keep the next
// row on its way.
inline NormShape norm_shape(int64_t pieces, bool grad) {
    const int64_t units = (pieces + 63) / 64;
    int waves = 1, chunks = units <= 1 ? 1 : 2;
    const int lanes = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    while (waves * chunks < units && waves < 16) waves = waves < 4 ? waves + 1 : waves % 3 ? waves / 2 * 3 : waves / 3 * 4;
    while (waves * chunks < units) ++chunks;
    return {waves, chunks, norm_teams(waves, grad), lanes};
}
constexpr int NORM_SUM_COLS = 32;    // columns of a workgroup that joins partial sums
hipError_t norm_forward_f32(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream);
hipError_t norm_forward_f16(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream);
hipError_t norm_forward_bf16(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream);
hipError_t norm_grad_f32(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream);
hipError_t norm_grad_f16(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream);
hipError_t norm_grad_bf16(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream);
// dweight[j] (dbias[j]) = the sum of `count` partial sums; nullptr: left out.
hipError_t norm_join(const float *part, int count, int N, float *dweight, float *dbias, hipStream_t stream);

// Routing of rows to experts (route.hip).  A row belongs to `lanes` lanes (16, 32 or 64) of a wave
// with `per` experts each (lanes * per >= experts), in chunks of 16 bytes of logits dealt to the lanes in turn
// (Share).  Workgroup b takes rows b * block_rows .. + block_rows - 1.
constexpr int ROUTE_MAX_K = 16, ROUTE_MAX_EXPERTS = 1024, ROUTE_MAX_BLOCKS = 256;
struct RouteParams {
    const void *logits;      // rows x experts, ldl
    const uint8_t *mask;     // one per row, 0: left out; nullptr: none is
    int32_t *index;          // rows x k (gradient: read)
    float *weight;           // rows x k
    int32_t *order, *place;  // rows * k
    int32_t *offsets;        // experts + 1
    float *slope, *loss;     // experts, 1; nullptr: left out
    // gradient
    const float *dweight, *dloss;    // rows x k; 1 (nullptr: 0)
    void *dlogits;           // ldl
    // workspace: `stride` numbers of each expert, the workgroups' choices of it ((experts + 1) of them: the last
    // are the used rows) and their summed probabilities; 4 times a power of two, at least blocks
    int32_t *hist;
    float *psum;
    int rows, experts, k, ldl, normalize;
    int block_rows, blocks, stride;
};
struct RouteShape {
    int lanes, per;
};
// Waves of a choosing workgroup: 16, or 8 where its rows of sums would need too much LDS; and the rows that
// one workgroup routes alone, two rounds of its waves at most (block_rows with blocks == 1; us, alone and as several:
// 64 experts, 8 chosen, 96 rows 8.4 and 8.9, 192 rows 12.1 and 9.2; 512 experts 16 rows 9.3 and 10.2, 32 rows 15.8 and 9.8).
constexpr int route_waves(int width) { return width <= 256 ? 16 : 8; }
constexpr int route_one_rows(int waves, int lanes) { return 2 * waves * (64 / lanes); }
// Choice, weights and the workgroups' sums; with one workgroup everything.
hipError_t route_choose_f32(const RouteParams &p, RouteShape s, hipStream_t stream);
hipError_t route_choose_f16(const RouteParams &p, RouteShape s, hipStream_t stream);
hipError_t route_choose_bf16(const RouteParams &p, RouteShape s, hipStream_t stream);
// The rest for several workgroups: order, place, offsets, slope, loss.
hipError_t route_place(const RouteParams &p, hipStream_t stream);
hipError_t route_grad_f32(const RouteParams &p, RouteShape s, unsigned grid, hipStream_t stream);
hipError_t route_grad_f16(const RouteParams &p, RouteShape s, unsigned grid, hipStream_t stream);
hipError_t route_grad_bf16(const RouteParams &p, RouteShape s, unsigned grid, hipStream_t stream);

}  // namespace tge
