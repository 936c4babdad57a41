// What the host code of the grouped, the 4-bit and the layer products shares: limits, rules that
// choose kernels, and small helpers.
#pragma once
#include <stdint.h>
#include <string.h>

#include "../../include/gemm.h"

namespace tge {
namespace host {

constexpr int64_t LIM31 = (int64_t)1 << 31;
constexpr int64_t MAX_GROUPS = (int64_t)1 << 20;
constexpr int64_t MAX_GRID = (int64_t)1 << 23;   // workgroups of up to 512 threads, 2^32 threads in all
constexpr int GROUP_M = 8;                 // tile rows per raster group, as in plain plans

// The integer held by an enum field (C callers may store any int).
template <class E>
inline int bits(const E &e) {
    static_assert(sizeof(E) == sizeof(int), "C ABI enums are int-sized");
    int v;
    memcpy(&v, &e, sizeof v);
    return v;
}

inline bool in(int v, int lo, int hi) { return v >= lo && v <= hi; }

inline int elem_bytes(int t) { return t == GEMM_F16 || t == GEMM_BF16 ? 2 : 4; }

inline const char *type_name(int t) {
    return t == GEMM_F16 ? "f16" : t == GEMM_BF16 ? "bf16" : "f32";
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles of `bm` rows that `rows` rows in `groups` ranges can need at most: every non-empty
// range has one begun tile, and the other rows fill whole ones.
inline int64_t row_tiles(int64_t rows, int64_t groups, int64_t bm) {
    const int64_t n = rows < groups ? rows : groups;
    return n + (rows - n) / bm;
}

// Whether the 256-wide tiles (one workgroup per CU) beat the 128-wide ones (two): with rows enough
// to fill them and a few rounds of them.  Measured (bf16, B not transposed; 128 -> 256): 8192 x 4096
// x 4096 over 8 experts 310 -> 275 us, 4096 x 14336 x 4096 over 8 562 -> 490, 16384 x 8192 x 2048
// over 16 592 -> 475, 32768 x 2048 x 1024 over 64 189 -> 182; but 8192 x 2048 x 4096 over 16 even
// and 2048 x 8192 x 2048 over 2 75 -> 87.
// With one expert the number of tiles is known, and what counts is that the last round is nearly
// full: 4096 x 4096 x 4096 (256 tiles) 111 -> 96, 6144 x 2048 x 4096 (192) 97 -> 83, 7168 x 4096 x
// 4096 (448) 203 -> 171; but 5120 x 4096 x 4096 (320) 148 -> 158.
inline bool rounds_full(int64_t wide_tiles) { return wide_tiles > 0 && 4 * wide_tiles >= 3 * 256 * ceil_div(wide_tiles, 256); }
// Sums below 512 leave them mostly storing, which the other tiles overlap: 8192 x 8192 over 4, K 128, 41 ->
// 54, K 256 58 -> 66, K 512 82 -> 89 (32768 x 8192 over 8: 161 -> 165, 216 -> 208, 338 -> 296).  With the
// gate, which reads C, 16384 x 8192 x 2048 over 16 683 -> 604 (614 -> 492 without it in the same run).
inline bool wide_tiles_pay(int64_t rows, int64_t groups, int64_t n, int64_t avg, int64_t N, int64_t K) {
    if (avg < 512 || K < 512) return false;
    if (groups == 1) return rounds_full(ceil_div(rows, 256) * ceil_div(N, 256));
    return ((double)rows / 256 + 0.5 * (double)n) * (double)ceil_div(N, 256) >= 384;
}

inline bool aligned(const void *p, uintptr_t to) { return (uintptr_t)p % to == 0; }

}  // namespace host
}  // namespace tge
