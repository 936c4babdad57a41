// What the host code of the grouped and the 4-bit products shares: limits and small helpers.
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

inline bool aligned(const void *p, uintptr_t to) { return (uintptr_t)p % to == 0; }

}  // namespace host
}  // namespace tge
