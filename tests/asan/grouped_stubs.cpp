// Host-only stand-ins for the kernels of the grouped and 4-bit products, so that their plan and run
// logic can be built and driven under the sanitizers on a machine with no GPU.  A launch checks
// what the kernels rely on and records itself instead of running.
#include <cstdio>
#include <cstdlib>

#include "../../tiled_gemm_epilogues_amd/csrc/gemm_internal.h"

namespace tge {
int grouped_launches = 0;
unsigned grouped_last_grid = 0;

namespace {
void require(bool ok, const char *what) {
    if (ok) return;
    std::fprintf(stderr, "stub launch: %s\n", what);
    std::abort();
}
template <int BM, int BN>
hipError_t launch(const GroupedParams &p, unsigned grid, hipStream_t) {
    require(p.offs != nullptr && (p.D != nullptr || (p.colsum && p.tiles_m == 0)), "pointers");
    require(p.tiles_n == (p.N + BN - 1) / BN, "column tiles");
    require(grid > 0 && grid < 1u << 23 && p.groups > 0 && p.rows >= 0, "sizes");
    require(!p.gate || (p.has_beta && p.C), "gate reads C");
    ++grouped_launches;
    grouped_last_grid = grid;
    return hipSuccess;
}
template <int BM, int BN>
const GroupedEntry *entry(const char *name) {
    static GroupedEntry e;
    e = {launch<BM, BN>, BM, BN, name};
    return &e;
}
hipError_t launch_quant(const QuantParams &p, unsigned grid, hipStream_t) {
    require(p.offs != nullptr || p.groups == 1, "offsets");
    require(grid > 0 && grid < 1u << 23 && p.block > 0 && p.K % p.block == 0, "sizes");
    require(p.block < 128 || p.block_rcp == (((uint64_t)1 << 32) + p.block / 128 - 1) / (p.block / 128), "reciprocal");
    ++grouped_launches;
    grouped_last_grid = grid;
    return hipSuccess;
}
const GroupedEntry *any(int mode, int op_b, int cfg) {
    if ((mode != GROUP_ROWS && mode != GROUP_K) || (mode == GROUP_K && op_b)) return nullptr;
    return cfg == CFG_128 ? entry<128, 128>("any128") : cfg == CFG_64 ? entry<64, 64>("any64") : nullptr;
}
const GroupedEntry *fast(int mode, int op_b, int tile, int rs) {
    if ((mode != GROUP_ROWS && mode != GROUP_K) || (mode == GROUP_K && op_b) || (rs && tile == 256)) return nullptr;
    return tile == 256 ? entry<256, 256>("fast256") : tile == 128 ? entry<128, 128>(rs ? "rs" : "fast128")
           : tile == 64 ? entry<64, 64>(rs ? "rs64" : "fast64") : nullptr;
}
const GroupedEntry *rows16(int op_b, int cg) {
    return cg == 4 ? entry<16, 64>("rows16") : cg == 1 && op_b == 1 ? entry<16, 16>("rows16")
           : cg == 2 && op_b == 0 ? entry<16, 32>("rows16") : nullptr;
}
const QuantEntry *qrows(int block, int cg) {
    static const QuantEntry e[2] = {{launch_quant, 16, 16, "qrows"}, {launch_quant, 16, 64, "qrows"}};
    return block == 32 || block == 64 || block == 128 ? &e[cg == 4] : nullptr;
}
const QuantEntry *qtile(int block) {
    static const QuantEntry e = {launch_quant, 128, 128, "qtile"};
    return block == 32 || block == 64 || block == 128 ? &e : nullptr;
}
}  // namespace

const GroupedEntry *grouped_any_f32_f32(int m, int b, int c) { return any(m, b, c); }
const GroupedEntry *grouped_any_f16_f16(int m, int b, int c) { return any(m, b, c); }
const GroupedEntry *grouped_any_f16_f32(int m, int b, int c) { return any(m, b, c); }
const GroupedEntry *grouped_any_bf16_bf16(int m, int b, int c) { return any(m, b, c); }
const GroupedEntry *grouped_any_bf16_f32(int m, int b, int c) { return any(m, b, c); }
const GroupedEntry *grouped_fast_f16_f16(int m, int b, int t, int r) { return fast(m, b, t, r); }
const GroupedEntry *grouped_fast_f16_f32(int m, int b, int t, int r) { return fast(m, b, t, r); }
const GroupedEntry *grouped_fast_bf16_bf16(int m, int b, int t, int r) { return fast(m, b, t, r); }
const GroupedEntry *grouped_fast_bf16_f32(int m, int b, int t, int r) { return fast(m, b, t, r); }
const GroupedEntry *grouped_rows16_f16_f16(int b, int c) { return rows16(b, c); }
const GroupedEntry *grouped_rows16_f16_f32(int b, int c) { return rows16(b, c); }
const GroupedEntry *grouped_rows16_bf16_bf16(int b, int c) { return rows16(b, c); }
const GroupedEntry *grouped_rows16_bf16_f32(int b, int c) { return rows16(b, c); }
const QuantEntry *quant_rows_f16_f16(int b, int c) { return qrows(b, c); }
const QuantEntry *quant_rows_f16_f32(int b, int c) { return qrows(b, c); }
const QuantEntry *quant_rows_bf16_bf16(int b, int c) { return qrows(b, c); }
const QuantEntry *quant_rows_bf16_f32(int b, int c) { return qrows(b, c); }
const QuantEntry *quant_tile_f16_f16(int b) { return qtile(b); }
const QuantEntry *quant_tile_f16_f32(int b) { return qtile(b); }
const QuantEntry *quant_tile_bf16_bf16(int b) { return qtile(b); }
const QuantEntry *quant_tile_bf16_f32(int b) { return qtile(b); }
}  // namespace tge
