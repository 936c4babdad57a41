// Device-side building blocks shared by the GEMM kernels (gfx950): element-type traits with
// their MFMA step, unaligned 16-byte loads, the XCD-aware tile scheduler and the fused
// register epilogue.  Included only by the kernel translation units.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_internal.h"

namespace tge {
namespace dev {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---- element types ---------------------------------------------------------------------------
// Every MFMA step consumes 16 bytes of K per lane for each operand: 8 fp16/bf16, 16 int8, or
// 4 fp32 (4 chained 32x32x2 instructions).

struct TF16 {
    static constexpr int E = 2;
    using acc_t = float;
    using accv_t = f32x16;
    using accv16_t = f32x4;
    __device__ static accv_t mma(u32x4 a, u32x4 b, accv_t c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    // 16x16 output, K = 32 per step (8 values per lane and operand, as above)
    __device__ static accv16_t mma16(u32x4 a, u32x4 b, accv16_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};
struct TBF16 {
    static constexpr int E = 2;
    using acc_t = float;
    using accv_t = f32x16;
    using accv16_t = f32x4;
    __device__ static accv_t mma(u32x4 a, u32x4 b, accv_t c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    __device__ static accv16_t mma16(u32x4 a, u32x4 b, accv16_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
struct TI8 {
    static constexpr int E = 1;
    using acc_t = int;
    using accv_t = i32x16;
    using accv16_t = i32x4;
    __device__ static accv_t mma(u32x4 a, u32x4 b, accv_t c) {
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                                     __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
    }
    // 16x16 output, K = 64 per step (16 values per lane and operand)
    __device__ static accv16_t mma16(u32x4 a, u32x4 b, accv16_t c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                     __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
    }
};
struct TF32 {
    static constexpr int E = 4;
    using acc_t = float;
    using accv_t = f32x16;
    // lanes 0-31 and 32-63 each supply 4 consecutive k; instruction j takes element j of both,
    // so the 4 instructions together cover 8 distinct k exactly once.
    __device__ static accv_t mma(u32x4 a, u32x4 b, accv_t c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // copy the element out first: bit_cast of a vector-element lvalue reads element 0
            const uint32_t aj = a[j], bj = b[j];
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__builtin_bit_cast(float, aj),
                                                     __builtin_bit_cast(float, bj), c, 0, 0, 0);
        }
        return c;
    }
    using accv16_t = f32x4;
    // 16x16 output: the 16 lanes of a group supply 4 consecutive k, the groups 16 in all
    __device__ static accv16_t mma16(u32x4 a, u32x4 b, accv16_t c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t aj = a[j], bj = b[j];
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, aj),
                                                     __builtin_bit_cast(float, bj), c, 0, 0, 0);
        }
        return c;
    }
};

// output element types
struct OF16 { using T = _Float16; static constexpr int E = 2; };
struct OBF16 { using T = __bf16; static constexpr int E = 2; };
struct OF32 { using T = float; static constexpr int E = 4; };
struct OI32 { using T = int; static constexpr int E = 4; };

// ---- small helpers ---------------------------------------------------------------------------

// 16-byte global load with no alignment requirement (gfx950 serves unaligned dwordx4 loads).
__device__ __forceinline__ u32x4 ldg16(const uint8_t *p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// Element-wise 16-byte chunk load: elements with index e < nvalid are read, the rest are 0.
template <int E>
__device__ __forceinline__ u32x4 ldg16_partial(const uint8_t *p, int nvalid) {
    uint8_t tmp[16];
#pragma unroll
    for (int e = 0; e < 16 / E; ++e) {
        if (e < nvalid) {
#pragma unroll
            for (int b = 0; b < E; ++b) tmp[e * E + b] = p[e * E + b];
        } else {
#pragma unroll
            for (int b = 0; b < E; ++b) tmp[e * E + b] = 0;
        }
    }
    u32x4 v;
    __builtin_memcpy(&v, tmp, 16);
    return v;
}

// Elements k .. k+7 of a row of K >= 8 two-byte elements, zero past its end: a whole load that ends
// with the row at the latest, moved down.
__device__ __forceinline__ u32x4 ldg16_row_end(const uint8_t *row, int k, int K) {
    const int at = min(k, K - 8), past = k - at;
    u32x4 v = ldg16(row + 2 * (int64_t)at);
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    if (past >= 4) {
        lo = hi;
        hi = 0;
    }
    const int n = 16 * (past & 3);
    lo = (lo >> n) | (n ? hi << (64 - n) : 0);
    hi >>= n;
    if (past >= 8) lo = 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// Transpose a VE x VE block of E-byte elements held as VE rows of 16 bytes.
template <int E>
__device__ __forceinline__ void transpose_block(const u32x4 *in, u32x4 *out);

template <>
__device__ __forceinline__ void transpose_block<2>(const u32x4 *in, u32x4 *out) {
    // out[e] word w = (in[2w] half e, in[2w+1] half e)
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t lo = in[2 * w][e >> 1], hi = in[2 * w + 1][e >> 1];
            // v_perm_b32: bytes 0-3 select from the second operand, 4-7 from the first
            out[e][w] = __builtin_amdgcn_perm(hi, lo, (e & 1) ? 0x07060302u : 0x05040100u);
        }
}

template <>
__device__ __forceinline__ void transpose_block<4>(const u32x4 *in, u32x4 *out) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r) out[e][r] = in[r][e];
}

template <>
__device__ __forceinline__ void transpose_block<1>(const u32x4 *in, u32x4 *out) {
    // out[e] byte r = in[r] byte e.  First gather 4 rows' byte e into one word with two
    // permutes per word.
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int wsel = e >> 2, bsel = e & 3;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t x0 = in[4 * w + 0][wsel], x1 = in[4 * w + 1][wsel];
            uint32_t x2 = in[4 * w + 2][wsel], x3 = in[4 * w + 3][wsel];
            // pick byte bsel of x0 (low) and x1 (next), then of x2, x3
            uint32_t s01 = __builtin_amdgcn_perm(x1, x0, (uint32_t)(bsel | ((bsel + 4) << 8)) | 0x0c0c0000u);
            uint32_t s23 = __builtin_amdgcn_perm(x3, x2, (uint32_t)(bsel | ((bsel + 4) << 8)) | 0x0c0c0000u);
            out[e][w] = (s01 & 0xffffu) | (s23 << 16);
        }
    }
}

// XCD-aware re-mapping: the hardware hands workgroup w to XCD w % 8.  Give each XCD a
// contiguous range of logical tile ids so the tiles resident on one XCD share its L2.
__device__ __forceinline__ int xcd_remap(int wg, int nwg) {
    constexpr int NX = 8;
    int q = nwg / NX, r = nwg % NX;
    int x = wg % NX, i = wg / NX;
    return (x < r) ? x * (q + 1) + i : r * (q + 1) + (x - r) * q + i;
}

// Load transform GEMM_TRANSFORM_RELU on a 16-byte chunk of E-byte elements: every element whose
// sign bit is set becomes +0 (max(x, 0) for every non-NaN x; the same rule for fp16, bf16 and
// int8 as 16- or 8-bit two's-complement sign tests, and for fp32 / int32 as 32-bit ones).
// Branch-free with the enable `on` (uniform 0/1), so it can sit inside a software pipeline.
template <int E>
__device__ __forceinline__ u32x4 zero_negative(u32x4 v, int on) {
    if constexpr (E == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (on && (int)v[i] < 0) ? 0u : v[i];
    } else if constexpr (E == 2) {
        typedef short s2 __attribute__((ext_vector_type(2)));
        const short fl = on ? (short)0 : (short)-32768;   // max(x, -32768) leaves x unchanged
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = v[i];   // bit_cast of a vector-element lvalue would read element 0
            const s2 h = __builtin_bit_cast(s2, w);
            v[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(h, (s2){fl, fl}));
        }
    } else {
        // sign bits m (0x80 per negative byte) -> whole-byte masks m | (m - m/128); no byte
        // borrows from its neighbour because each byte of m is >= the same byte of m >> 7
        const uint32_t sel = on ? 0x80808080u : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t m = v[i] & sel;
            v[i] &= ~(m | (m - (m >> 7)));
        }
    }
    return v;
}

// A C element as the epilogue uses it: in the accumulation type, with the load transform
// (relu_in: sign bit set -> +0) applied.
template <class T>
__device__ __forceinline__ float c_in_f(T c, int relu_in) {
    const float f = (float)c;
    return (relu_in && __builtin_bit_cast(int, f) < 0) ? 0.0f : f;
}
__device__ __forceinline__ int c_in_i(int c, int relu_in) { return (relu_in && c < 0) ? 0 : c; }

// Strided batch: workgroup id -> (product b, id inside the product, `per` ids per product); the
// operand pointers of `p` are moved to product b.  Consecutive ids share a product, so the
// XCD-contiguous id ranges of xcd_remap keep each product on few XCDs.  With two batch modes
// product b is (b1, b2) = (b / batch2, b % batch2), moved by b1 * stride + b2 * stride2: the
// index map of a tensor contraction whose batch index has two modes with their own strides.
template <int EAB, int ECD>
__device__ __forceinline__ int select_batch(GemmParams &p, int id, int per) {
    const int b = __builtin_amdgcn_readfirstlane(id / per);   // uniform: keeps pointers scalar
    if (b > 0) {
        const int b1 = __builtin_amdgcn_readfirstlane(b / p.batch2);
        const int b2 = b - b1 * p.batch2;
        const int64_t oa = b1 * p.stride_a + b2 * p.stride2_a, ob = b1 * p.stride_b + b2 * p.stride2_b;
        const int64_t oc = b1 * p.stride_c + b2 * p.stride2_c, obias = b1 * p.stride_bias + b2 * p.stride2_bias;
        p.A = static_cast<const uint8_t *>(p.A) + oa * EAB;
        p.B = static_cast<const uint8_t *>(p.B) + ob * EAB;
        if (p.C) p.C = static_cast<const uint8_t *>(p.C) + oc * ECD;
        p.D = static_cast<uint8_t *>(p.D) + oc * ECD;
        if (p.bias) p.bias = static_cast<const uint8_t *>(p.bias) + obias * 4;
    }
    return __builtin_amdgcn_readfirstlane(id - b * per);
}

// Grouped raster: consecutive ids walk down group_m tile rows, then move one tile column.
__device__ __forceinline__ void raster(int id, int tiles_m, int tiles_n, int group_m, int &tm, int &tn) {
    int per_group = group_m * tiles_n;
    int g = id / per_group;
    int first = g * group_m;
    int gm = min(tiles_m - first, group_m);
    int in = id - g * per_group;
    tm = first + in % gm;
    tn = in / gm;
}

// ---- groups ----------------------------------------------------------------------------------

template <int GRP>
using ParamsOf = typename std::conditional<GRP == GROUP_NONE, GemmParams,
                 typename std::conditional<GRP == GROUP_LAYER, LayerParams, GroupedParams>::type>::type;

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}
// The base of a grouped kernel's direct-to-LDS loads, which take it from scalar registers.  Only
// for those: ordinary loads through a pointer rebuilt from its halves would be flat loads, which
// also wait for LDS.
template <int GRP>
__device__ __forceinline__ const uint8_t *dma_base(const void *q) {
    if constexpr (GRP == GROUP_NONE) return static_cast<const uint8_t *>(q);
    else return reinterpret_cast<const uint8_t *>(uniform64(reinterpret_cast<int64_t>(q)));
}

// Range e of the offsets, clamped to [0, rows] and never negative.
__device__ __forceinline__ void group_range(const GroupedParams &p, int e, int &lo, int &hi) {
    lo = min(max(p.offs[e], 0), p.rows);
    hi = max(min(p.offs[e + 1], p.rows), lo);
}

// Inclusive scans over the wave's 64 lanes (values >= 0), with the data-parallel lane moves: a
// shift by 1, 2, 4, 8 inside each row of 16 lanes, then the last lane of rows 0 and 2 into rows 1
// and 3, then lane 31 into rows 2 and 3.  Lanes without a source keep 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ int lane_move(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_scan_add(int v) {
    v += lane_move<0x111, 0xf>(v);
    v += lane_move<0x112, 0xf>(v);
    v += lane_move<0x114, 0xf>(v);
    v += lane_move<0x118, 0xf>(v);
    v += lane_move<0x142, 0xa>(v);
    v += lane_move<0x143, 0xc>(v);
    return v;
}
// Sum of the wave's 64 values, the same in every lane (scalar), by the same moves.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_moved(float v) {
    return v + __builtin_bit_cast(float, lane_move<CTRL, ROWS>(__builtin_bit_cast(int, v)));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = add_moved<0x111, 0xf>(v);
    v = add_moved<0x112, 0xf>(v);
    v = add_moved<0x114, 0xf>(v);
    v = add_moved<0x118, 0xf>(v);
    v = add_moved<0x142, 0xa>(v);
    v = add_moved<0x143, 0xc>(v);
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
// v of another lane.  MOVE: a data-parallel move inside 16 lanes (N on in their ring; mirrored in 8 lanes; the
// neighbour, or two on, in 4), or 16 or 32: the lane that far away.
constexpr int RING = 0x120, MIRROR_8 = 0x141, NEXT_OF_2 = 0xb1, OTHER_2 = 0x4e;
template <int MOVE>
__device__ __forceinline__ int moved(int v) {
    if constexpr (MOVE == 16) return __builtin_amdgcn_ds_swizzle(v, 0x401f);
    else if constexpr (MOVE == 32) return __shfl_xor(v, 32);
    else return __builtin_amdgcn_update_dpp(0, v, MOVE, 0xf, 0xf, true);
}
// f(move) for the moves after each of which twice as many of the LANES lanes have been joined.
template <int LANES, class F>
__device__ __forceinline__ void lane_steps(F f) {
    if constexpr (LANES == 8) {
        f(std::integral_constant<int, MIRROR_8>());
        f(std::integral_constant<int, NEXT_OF_2>());
        f(std::integral_constant<int, OTHER_2>());
    } else {
        f(std::integral_constant<int, RING + 8>());
        f(std::integral_constant<int, RING + 4>());
        f(std::integral_constant<int, RING + 2>());
        f(std::integral_constant<int, RING + 1>());
        if constexpr (LANES >= 32) f(std::integral_constant<int, 16>());
        if constexpr (LANES >= 64) f(std::integral_constant<int, 32>());
    }
}

// Sum over LANES lanes side by side, in each of them.
template <int LANES>
__device__ __forceinline__ float side_sum(float v) {
    if constexpr (LANES == 64) return wave_sum(v);
    lane_steps<LANES>([&](auto move) { v += __builtin_bit_cast(float, moved<move.value>(__builtin_bit_cast(int, v))); });
    return v;
}
__device__ __forceinline__ int wave_scan_max(int v) {
    v = max(v, lane_move<0x111, 0xf>(v));
    v = max(v, lane_move<0x112, 0xf>(v));
    v = max(v, lane_move<0x114, 0xf>(v));
    v = max(v, lane_move<0x118, 0xf>(v));
    v = max(v, lane_move<0x142, 0xa>(v));
    v = max(v, lane_move<0x143, 0xc>(v));
    return v;
}

// The ranges e0 .. e0+63, one per lane, with their tiles of bm rows: starts are the running
// maximum of the clamped offsets (ordered offsets are their own), so that the ranges never overlap
// and the launch's bound on the number of tiles holds for any offsets.  `carry`: the maximum
// before e0, moved on.
struct RangeChunk {
    int lo, hi, mine, incl;   // the lane's range, its tiles, and the tiles of lanes 0 .. lane
};
__device__ __forceinline__ RangeChunk range_chunk(const GroupedParams &p, int e0, int bm, int &carry) {
    const int e = e0 + (int)(threadIdx.x & 63);
    const bool in = e < p.groups;
    // lanes past the last range read the last offset: both loads are in flight together
    const int a = p.offs[min(e, p.groups)], b = p.offs[min(e + 1, p.groups)];
    RangeChunk c;
    c.lo = max(wave_scan_max(min(max(a, 0), p.rows)), carry);
    c.hi = max(min(b, p.rows), c.lo);
    carry = __builtin_amdgcn_readlane(c.hi, 63);
    c.mine = in ? (c.hi - c.lo + bm - 1) / bm * p.tiles_n : 0;
    c.incl = wave_scan_add(c.mine);
    return c;
}

// GROUP_ROWS: workgroup wg -> an expert, bm of its rows and a column tile.  The launch has a
// workgroup for every tile that `rows` rows in `groups` ranges can need; the real count is known
// from the offsets, read here by every wave (64 ranges at a time, one per lane): a workgroup past
// it has no tile (false).  The tiles of one expert are consecutive and each XCD takes a contiguous
// run of them, so an expert's weights stay with few XCDs' L2.  On return the pointers stand at
// the tile's first row (so that 32-bit offsets inside the tile are enough however long A and D
// are; the selection costs nothing measurable up to 64 ranges, 0.5 us at 128 and 7 us at 1024),
// p.M is the number of the expert's rows from there on, and tn the column tile; `expert`,
// where given, receives the expert.
template <int EAB, int ECD>
__device__ __forceinline__ bool select_rows(GroupedParams &p, int wg, int bm, int &tn, int *expert = nullptr) {
    int carry = 0, total = 0, e0 = 0;
    RangeChunk c;
    for (;; e0 += 64) {
        c = range_chunk(p, e0, bm, carry);
        total += __builtin_amdgcn_readlane(c.incl, 63);
        if (e0 + 64 >= p.groups) break;
    }
    if (wg >= total) return false;
    int id = xcd_remap(wg, total);
    if (p.groups > 64) {   // more than one chunk: find the one that holds id
        carry = 0;
        for (e0 = 0;; e0 += 64) {
            c = range_chunk(p, e0, bm, carry);
            const int n = __builtin_amdgcn_readlane(c.incl, 63);
            if (id < n) break;
            id -= n;
        }
    }
    const int src = __ffsll((unsigned long long)__ballot(c.incl > id)) - 1;   // id < the chunk's tiles
    id -= __builtin_amdgcn_readlane(c.incl, src) - __builtin_amdgcn_readlane(c.mine, src);
    const int lo = __builtin_amdgcn_readlane(c.lo, src), hi = __builtin_amdgcn_readlane(c.hi, src);
    const int e = e0 + src;
    if (expert) *expert = e;
    int tm;
    raster(id, (hi - lo + bm - 1) / bm, p.tiles_n, p.group_m, tm, tn);
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    const int64_t row = lo + (int64_t)tm * bm;
    p.M = __builtin_amdgcn_readfirstlane(hi - (int)row);
    p.A = static_cast<const uint8_t *>(p.A) + uniform64(row * p.lda * EAB);
    p.B = static_cast<const uint8_t *>(p.B) + uniform64(e * p.stride_b * EAB);
    if (p.C) p.C = static_cast<const uint8_t *>(p.C) + row * p.ldc * ECD;
    p.D = static_cast<uint8_t *>(p.D) + row * p.ldc * ECD;
    if (p.bias) p.bias = static_cast<const uint8_t *>(p.bias) + e * p.stride_bias * 4;
    return true;
}

// GROUP_LAYER: as GROUP_ROWS, Z moved with D; without offsets the tiles of one product.
template <int EAB, int ECD>
__device__ __forceinline__ bool select_layer(LayerParams &p, int wg, int bm, int &tn) {
    int64_t moved;
    if (p.offs) {
        const uint8_t *d = static_cast<const uint8_t *>(p.D);
        if (!select_rows<EAB, ECD>(p, wg, bm, tn)) return false;
        moved = static_cast<const uint8_t *>(p.D) - d;
    } else {
        int tm;
        raster(xcd_remap(wg, p.tiles_m * p.tiles_n), p.tiles_m, p.tiles_n, p.group_m, tm, tn);
        tm = __builtin_amdgcn_readfirstlane(tm);
        tn = __builtin_amdgcn_readfirstlane(tn);
        const int64_t row = (int64_t)tm * bm;
        p.M = __builtin_amdgcn_readfirstlane(p.rows - (int)row);
        p.A = static_cast<const uint8_t *>(p.A) + uniform64(row * p.lda * EAB);
        moved = row * p.ldc * ECD;
        if (p.C) p.C = static_cast<const uint8_t *>(p.C) + moved;
        p.D = static_cast<uint8_t *>(p.D) + moved;
    }
    if (p.Z) p.Z = static_cast<uint8_t *>(p.Z) + moved;
    return true;
}

// GROUP_K: workgroup id -> a product and a tile of it.  All products have the same tiles; the
// tiles of one product are spread over the XCDs in contiguous runs (the ranges' lengths differ,
// so whole products per XCD would leave some XCDs with the long ones).
template <int EAB, int ECD>
__device__ __forceinline__ void select_k(GroupedParams &p, int id, int &tm, int &tn) {
    const int per = p.tiles_m * p.tiles_n;
    const int e = __builtin_amdgcn_readfirstlane(id / per);
    int lo, hi;
    group_range(p, e, lo, hi);
    raster(xcd_remap(id - e * per, per), p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    tm = __builtin_amdgcn_readfirstlane(tm);
    tn = __builtin_amdgcn_readfirstlane(tn);
    p.K = __builtin_amdgcn_readfirstlane(hi - lo);
    p.A = static_cast<const uint8_t *>(p.A) + uniform64((int64_t)lo * p.lda * EAB);
    p.B = static_cast<const uint8_t *>(p.B) + uniform64((int64_t)lo * p.ldb * EAB);
    if (p.C) p.C = static_cast<const uint8_t *>(p.C) + e * p.stride_c * ECD;
    p.D = static_cast<uint8_t *>(p.D) + e * p.stride_c * ECD;
}

// GROUP_K: the column sums of B over one range (the gradient of a bias added to its rows), as
// extra workgroups of 256 threads in front of the products': COLSUM_COLS columns of one range, 32
// rows at a time, eight times in flight; the 32 partial sums of a column are added through `part`
// (256 x 8 floats of LDS).  Sums are in fp32 and in a fixed order.  They read B once more, hidden
// beside the products: 16384 rows, 16 experts of 4096 x 2048, 365 us without and 371 with them; 32768
// rows, one expert of 4096 x 4096 (one full round of 256-wide tiles), 778 and 857 (in two rounds of
// 128-wide ones 987 and 1067; with 128 columns, 16 rows four times in flight 1223).
template <class T>
__device__ __forceinline__ void colsum_block(const GroupedParams &p, int id, float *part) {
    constexpr int LPR = COLSUM_COLS / 8, ROWS = 256 / LPR;   // threads per row, rows at a time
    const int nb = (p.N + COLSUM_COLS - 1) / COLSUM_COLS;
    const int e = id / nb, tid = threadIdx.x;
    const int n = (id - e * nb) * COLSUM_COLS + (tid % LPR) * 8;
    int lo, hi;
    group_range(p, e, lo, hi);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    const T *B = static_cast<const T *>(p.B);
    if (n + 8 <= p.N) {
#pragma unroll 8
        for (int r = lo + tid / LPR; r < hi; r += ROWS) {
            T v[8];
            __builtin_memcpy(v, B + (int64_t)r * p.ldb + n, sizeof(v));
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += (float)v[i];
        }
    } else if (n < p.N) {   // columns past N read the last one; they are not stored
#pragma unroll 2
        for (int r = lo + tid / LPR; r < hi; r += ROWS)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += (float)B[(int64_t)r * p.ldb + min(n + i, p.N - 1)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[tid * 8 + i] = s[i];
    __syncthreads();
    if (tid < COLSUM_COLS) {
        const int col = (id - e * nb) * COLSUM_COLS + tid;
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) t += part[(r * LPR + (tid >> 3)) * 8 + (tid & 7)];
        if (col < p.N) p.colsum[(int64_t)e * p.N + col] = t;
    }
}
// how many of them a launch has
__device__ __forceinline__ int colsum_blocks(const GroupedParams &p) {
    return p.colsum ? p.groups * ((p.N + COLSUM_COLS - 1) / COLSUM_COLS) : 0;
}

// ---- epilogue --------------------------------------------------------------------------------

// Epilogue of a wave's MFMA tiles.  Lane l holds, for 32x32 tile (i, j), accumulator register
// 4g+e = D[mbase + 32i + l%32][nbase + 32j + 8g + 4(l/32) + e].  The bias values of the wave's
// columns are loaded once, the C values of one 32-row block are loaded together before any of
// its stores (C == D is allowed: every element is read before the same lane writes it), so the
// loads overlap instead of each waiting for the store before it.
// gate (float outputs): D = C > 0 ? alpha * acc : 0 in place of the sum with beta * C.
template <class O, class Acc, class AccV, int TM, int TN>
__device__ __forceinline__ void store_tile(const GemmParams &p, int mbase, int nbase, int lane,
                                           AccV (&acc)[TM][TN], const bool gate = false) {
    using T = typename O::T;
    constexpr bool INT = std::is_same<Acc, int>::value;
    using B = typename std::conditional<INT, int, float>::type;
    const int hi = lane >> 5, rl = lane & 31;
    const int N = p.N;
    const bool full_n = nbase + 32 * TN <= N;
    const B *bias = static_cast<const B *>(p.bias);
    const T *C = static_cast<const T *>(p.C);
    T *D = static_cast<T *>(p.D);

    B bv[TN][4][4];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int n = nbase + 32 * j + 8 * g + 4 * hi;
            if (p.has_bias && full_n) {
                __builtin_memcpy(bv[j][g], bias + n, sizeof(bv[j][g]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) bv[j][g][e] = (p.has_bias && n + e < N) ? bias[n + e] : (B)0;
            }
        }

#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = mbase + 32 * i + rl;
        if (m >= p.M) continue;
        const int64_t row = (int64_t)m * p.ldc;
        T cv[TN][4][4];
        if (p.has_beta) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = nbase + 32 * j + 8 * g + 4 * hi;
                    if (full_n) {
                        __builtin_memcpy(cv[j][g], C + row + n, sizeof(cv[j][g]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) cv[j][g][e] = (n + e < N) ? C[row + n + e] : (T)0;
                    }
                }
        }
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int n = nbase + 32 * j + 8 * g + 4 * hi;
                T out[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (INT) {
                        // integer path: alpha == 1, beta in {0, 1}
                        int t = acc[i][j][4 * g + e] + bv[j][g][e];
                        if (p.has_beta) t += c_in_i((int)cv[j][g][e], p.xform_c);
                        if (p.relu) t = t > 0 ? t : 0;
                        out[e] = (T)t;
                    } else {
                        float t = p.alpha * acc[i][j][4 * g + e];
                        if (gate) t = (float)cv[j][g][e] > 0.0f ? t : 0.0f;
                        else if (p.has_beta) t += p.beta * c_in_f(cv[j][g][e], p.xform_c);
                        t += bv[j][g][e];
                        if (p.relu) t = t > 0.0f ? t : 0.0f;
                        out[e] = (T)t;
                    }
                }
                if (full_n) {
                    __builtin_memcpy(D + row + n, out, sizeof(out));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < N) D[row + n + e] = out[e];
                }
            }
    }
}

}  // namespace dev
}  // namespace tge
