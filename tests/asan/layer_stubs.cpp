// Host-only stand-ins for the kernels of a layer's products, layer norm and routing, so that their plan
// and run logic can be built and driven under the sanitizers on a machine with no GPU.  A launch
// checks what the kernels rely on and records itself instead of running.
#include <cstdio>
#include <cstdlib>

#include "../../tiled_gemm_epilogues_amd/csrc/gemm_internal.h"

namespace tge {
int layer_launches = 0, norm_launches = 0, route_launches = 0;

namespace {
void require(bool ok, const char *what) {
    if (ok) return;
    std::fprintf(stderr, "stub launch: %s\n", what);
    std::abort();
}
bool whole(const void *p, uintptr_t to) { return p && (uintptr_t)p % to == 0; }

enum { ANY, DIRECT, STAGED, ROWS };
template <int BM, int BN, int KIND, int OPB, int ES>
hipError_t launch(const LayerParams &p, unsigned grid, hipStream_t) {
    require(whole(p.D, ES) && (p.K == 0 || (whole(p.A, ES) && whole(p.B, ES))), "pointers");
    require(p.tiles_n == (p.N + BN - 1) / BN && p.tiles_m == (p.rows + BM - 1) / BM, "tiles");
    require(grid > 0 && grid < 1u << 23 && p.groups > 0 && p.rows > 0 && p.M == p.rows, "sizes");
    require(p.offs || (p.groups == 1 && grid == (unsigned)(p.tiles_m * p.tiles_n)), "offsets");
    require(!p.grad || (p.Z && !p.has_beta && !p.has_bias && p.act != ACT_NONE), "gradient");
    require(!p.has_beta || p.C, "C");
    const int64_t line = (int64_t)p.lda * ES;
    if (KIND == DIRECT)
        require(p.K * ES >= 128 && whole(p.A, 16) && whole(p.B, 16) && p.lda * ES % 16 == 0 && p.ldb * ES % 16 == 0 &&
                    p.stride_b * ES % 16 == 0 && (OPB || p.N * ES % 16 == 0) && line * 256 < (int64_t)1 << 31, "direct loads");
    if (KIND == STAGED) require(p.K > 0 && p.N * ES >= 16 && line * 256 < (int64_t)1 << 31, "staged loads");
    if (KIND == ROWS) require(p.K * ES >= 16 && (OPB || p.N * ES >= 16) && line * 64 < (int64_t)1 << 31, "few rows");
    ++layer_launches;
    return hipSuccess;
}
template <int BM, int BN, int KIND, int OPB, int ES>
const LayerEntry *entry(const char *name) {
    static const LayerEntry e = {launch<BM, BN, KIND, OPB, ES>, BM, BN, name};
    return &e;
}
template <int BM, int BN, int KIND, int ES>
const LayerEntry *of(int op_b, const char *name) {
    return op_b ? entry<BM, BN, KIND, 1, ES>(name) : entry<BM, BN, KIND, 0, ES>(name);
}
template <int ES>
const LayerEntry *any(int op_b, int cfg) {
    return cfg == CFG_128 ? of<128, 128, ANY, ES>(op_b, "any128") : cfg == CFG_64 ? of<64, 64, ANY, ES>(op_b, "any64") : nullptr;
}
template <int ES>
const LayerEntry *fast(int op_b, int tile, int rs) {
    if (rs) return tile == 128 ? of<128, 128, STAGED, ES>(op_b, "rs") : tile == 64 ? of<64, 64, STAGED, ES>(op_b, "rs64") : nullptr;
    return tile == 256 ? of<256, 256, DIRECT, ES>(op_b, "fast256") : tile == 128 ? of<128, 128, DIRECT, ES>(op_b, "fast128")
           : tile == 64 ? of<64, 64, DIRECT, ES>(op_b, "fast64") : nullptr;
}
template <int BM, int ES>
const LayerEntry *rows_of(int op_b, int cg) {
    return cg == 4 ? of<BM, 64, ROWS, ES>(op_b, "rows") : cg == 1 && op_b ? entry<BM, 16, ROWS, 1, ES>("rows")
           : cg == 2 && !op_b ? entry<BM, 32, ROWS, 0, ES>("rows") : nullptr;
}
template <int ES>
const LayerEntry *rows(int op_b, int rt, int cg) {
    return rt == 1 ? rows_of<16, ES>(op_b, cg) : rt == 2 ? rows_of<32, ES>(op_b, cg) : rt == 4 ? rows_of<64, ES>(op_b, cg) : nullptr;
}

template <int ES>
hipError_t forward(const NormParams &p, NormShape s, unsigned grid, hipStream_t) {
    require(whole(p.X, ES) && whole(p.Y, ES) && p.rows > 0 && p.N > 0 && p.ldx >= p.N && p.ldy >= p.N, "norm operands");
    require(s.waves >= 1 && s.waves * s.teams <= 16 && s.waves * s.chunks * 1024 >= p.N * ES, "norm team");
    require(grid > 0 && grid <= (unsigned)p.rows && grid <= 1024 * 4, "norm grid");
    ++norm_launches;
    return hipSuccess;
}
template <int ES>
hipError_t gradient(const NormParams &p, NormShape s, unsigned grid, hipStream_t st) {
    require(whole(p.dX, ES) && p.mean && p.rstd && (!p.has_beta || whole(p.C, ES)) && grid <= 256, "norm gradient");
    return forward<ES>(p, s, grid, st);
}
template <int ES>
hipError_t choose(const RouteParams &p, RouteShape s, hipStream_t) {
    require(p.rows == 0 || (whole(p.logits, ES) && p.index && p.weight && p.order && p.place), "route operands");
    require(p.offsets && s.lanes * s.per >= p.experts && p.k <= 16 && p.k <= p.experts, "route sizes");
    require(p.blocks >= 1 && p.blocks <= ROUTE_MAX_BLOCKS && (int64_t)p.blocks * p.block_rows >= p.rows, "route blocks");
    require(p.blocks == 1 || (p.hist && p.psum && p.psum == (float *)(p.hist + (p.experts + 1) * p.stride) && p.stride >= p.blocks && p.stride <= ROUTE_MAX_BLOCKS &&
            (p.stride & (p.stride - 1)) == 0 && p.stride >= 4), "route workspace");
    ++route_launches;
    return hipSuccess;
}
template <int ES>
hipError_t route_gradient(const RouteParams &p, RouteShape s, unsigned grid, hipStream_t) {
    require(p.rows > 0 && whole(p.logits, ES) && whole(p.dlogits, ES) && (!p.dweight || p.index) && (!p.dloss || p.slope), "route gradient");
    require(grid > 0 && grid <= 2048 && s.lanes * s.per >= p.experts, "route grid");
    ++route_launches;
    return hipSuccess;
}
}  // namespace

const LayerEntry *layer_any_f32_f32(int b, int c) { return any<4>(b, c); }
const LayerEntry *layer_any_f16_f16(int b, int c) { return any<2>(b, c); }
const LayerEntry *layer_any_f16_f32(int b, int c) { return any<2>(b, c); }
const LayerEntry *layer_any_bf16_bf16(int b, int c) { return any<2>(b, c); }
const LayerEntry *layer_any_bf16_f32(int b, int c) { return any<2>(b, c); }
const LayerEntry *layer_fast_f32_f32(int b, int t, int r) { return fast<4>(b, t, r); }
const LayerEntry *layer_fast_f16_f16(int b, int t, int r) { return fast<2>(b, t, r); }
const LayerEntry *layer_fast_f16_f32(int b, int t, int r) { return fast<2>(b, t, r); }
const LayerEntry *layer_fast_bf16_bf16(int b, int t, int r) { return fast<2>(b, t, r); }
const LayerEntry *layer_fast_bf16_f32(int b, int t, int r) { return fast<2>(b, t, r); }
const LayerEntry *layer_rows_f32_f32(int b, int r, int c) { return rows<4>(b, r, c); }
const LayerEntry *layer_rows_f16_f16(int b, int r, int c) { return rows<2>(b, r, c); }
const LayerEntry *layer_rows_f16_f32(int b, int r, int c) { return rows<2>(b, r, c); }
const LayerEntry *layer_rows_bf16_bf16(int b, int r, int c) { return rows<2>(b, r, c); }
const LayerEntry *layer_rows_bf16_f32(int b, int r, int c) { return rows<2>(b, r, c); }

hipError_t norm_forward_f32(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return forward<4>(p, s, g, st); }
hipError_t norm_forward_f16(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return forward<2>(p, s, g, st); }
hipError_t norm_forward_bf16(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return forward<2>(p, s, g, st); }
hipError_t norm_grad_f32(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return gradient<4>(p, s, g, st); }
hipError_t norm_grad_f16(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return gradient<2>(p, s, g, st); }
hipError_t norm_grad_bf16(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return gradient<2>(p, s, g, st); }
hipError_t norm_join(const float *part, int count, int N, float *dw, float *db, hipStream_t) {
    require((part || count == 0) && count >= 0 && count <= 256 && N > 0 && (dw || db), "join");
    ++norm_launches;
    return hipSuccess;
}

hipError_t route_choose_f32(const RouteParams &p, RouteShape s, hipStream_t st) { return choose<4>(p, s, st); }
hipError_t route_choose_f16(const RouteParams &p, RouteShape s, hipStream_t st) { return choose<2>(p, s, st); }
hipError_t route_choose_bf16(const RouteParams &p, RouteShape s, hipStream_t st) { return choose<2>(p, s, st); }
hipError_t route_place(const RouteParams &p, hipStream_t) {
    require(p.blocks > 1 && p.hist && p.rows > 0, "place");
    ++route_launches;
    return hipSuccess;
}
hipError_t route_grad_f32(const RouteParams &p, RouteShape s, unsigned g, hipStream_t st) { return route_gradient<4>(p, s, g, st); }
hipError_t route_grad_f16(const RouteParams &p, RouteShape s, unsigned g, hipStream_t st) { return route_gradient<2>(p, s, g, st); }
hipError_t route_grad_bf16(const RouteParams &p, RouteShape s, unsigned g, hipStream_t st) { return route_gradient<2>(p, s, g, st); }
}  // namespace tge
