// A layer's products of few rows on gfx950, any alignment and any K: 16 * RT rows and 16 * CG columns of one
// expert (or of the one matrix) per workgroup, K divided over its 8 waves.  Bound by the weights' bytes,
// each read once per 16 * RT rows.
//
// Each wave takes its part of K in chunks of 128 or 256 bytes, loaded to registers and put into a private LDS slot that
// only changes the lane order.  DEPTH chunks are on their way while one is multiplied, and more rows
// share a chunk of B instead of reading it again.  Loads take few long pieces of rows rather than many
// short ones: whole 128- or 256-byte pieces of 8 or 4 rows.  (Rows are often a power of two apart, and so in
// one channel of the memory: with 64-byte pieces of 16 rows, 16 rows of 4096 x 16384 took 43 us, of 16384
// x 4096, the same bytes, 30.)  A B stored K x N is loaded in rows of 64 or 32 columns; 16-bit values are
// read with the transposing read, as in gemm_rows16.hip, fp32 ones (for which there is none) one by one.
//
// Preconditions (checked by the host): K of at least one 16-byte chunk, N too when B is not transposed, 64
// rows of A within 2^31 bytes.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"
#include "layer_epilogue.hpp"

namespace tge {
namespace {

using namespace dev;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int WAVES = 8;

// 16 rows of KB bytes of k, in LDS: 16-byte piece q of row r, at a place that differs for the 16 rows
// that a read takes one piece of (256 bytes are all banks), and that a whole load fills.
template <int KB>
__device__ __forceinline__ int piece(int r, int q) {
    return r * KB + ((q ^ (KB == 256 ? r & 15 : r >> 1 & 7)) << 4);
}

// Elements k .. k + 16 / E - 1 of a row of K, zero past its end: a whole load that ends with the row at the
// latest, moved down.
template <int E>
__device__ __forceinline__ u32x4 row_end(const uint8_t *row, int k, int K) {
    if constexpr (E == 2) {
        return ldg16_row_end(row, k, K);
    } else {
        const int at = min(k, K - 4), past = k - at;
        const u32x4 v = ldg16(row + 4 * (int64_t)at);
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x = 0;
#pragma unroll
            for (int j = i; j < 4; ++j) x = j - i == past ? v[j] : x;
            r[i] = x;
        }
        return r;
    }
}

// BT: B stored N x K; RT: groups of 16 rows; CG: groups of 16 columns; KB: bytes of k per chunk.
template <class TI, class TO, bool BT, int RT, int CG, int KB>
__global__ __launch_bounds__(WAVES * 64, 2) void layer_rows(LayerParams p) {
    using T = typename TO::T;
    static_assert(BT || ((CG == 4 || CG == 2) && KB == 128), "rows of 64 or 32 columns");
    constexpr int E = TI::E, VE = 16 / E, KC = KB / E;       // k per chunk
    constexpr int NI = KB / 64;                              // steps of 64 bytes of k, 16 to a lane group
    constexpr int LPR = CG * E, RPL = 64 / LPR;              // K x N: lanes per row, rows per load
    constexpr int NB = BT ? CG * NI : KC / RPL, NA = RT * NI;   // 1 KiB loads per chunk
    constexpr int COLS = 16 * CG, DEPTH = NA + NB > 12 ? 1 : 2;   // chunks on their way (the largest fill the registers)
    constexpr int OFF_A = NB * 1024, SLOT = OFF_A + NA * 1024;
    static_assert(SLOT >= RT * CG * 1024, "the slots hold the waves' sums at the end");
    __shared__ __attribute__((aligned(16))) uint8_t smem[WAVES * SLOT];

    int tn;
    if (!select_layer<E, (int)sizeof(T)>(p, blockIdx.x, 16 * RT, tn)) return;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int PPR = KB / 16, RPI = 64 / PPR;              // rows along K: pieces per row, rows per load
    const int lr = lane / PPR, lq = lane % PPR;              // load order: row, piece
    const int n0 = tn * COLS;
    const int nch = (p.K + KC - 1) / KC;
    const int c0 = (int)((int64_t)nch * wave / WAVES), c1 = (int)((int64_t)nch * (wave + 1) / WAVES);
    uint8_t *const slot = smem + wave * SLOT;
    const uint8_t *const A = static_cast<const uint8_t *>(p.A), *const B = static_cast<const uint8_t *>(p.B);
    // load i of A: rows RPI i + lr; past the range its last one (their results are not stored)
    uint32_t arow[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) arow[i] = (uint32_t)min(RPI * i + lr, p.M - 1) * (uint32_t)p.lda * (uint32_t)E;
    // BT: rows n0 + RPI i + lr of B.  Else: row lane / LPR of the load, VE columns from n0 + VE * (lane % LPR)
    uint32_t brow[BT ? NB : 1];
    const int br = lane / LPR, bq = lane % LPR, bc = n0 + VE * bq, bcol = min(bc, p.N - 1);
    if constexpr (BT) {
#pragma unroll
        for (int i = 0; i < NB; ++i) brow[i] = (uint32_t)min(n0 + RPI * i + lr, p.N - 1) * (uint32_t)p.ldb * (uint32_t)E;
    } else {
        brow[0] = ((uint32_t)br * (uint32_t)p.ldb + (uint32_t)bcol) * (uint32_t)E;
    }
    // (uniform) a chunk whose loads need no care: inside K; with columns past N also a row after it
    const int last = p.K - KC - (!BT && n0 + COLS > p.N ? 1 : 0);

    struct Chunk {
        u32x4 b[NB], a[NA];
    };
    // ONCE: weights that no other workgroup reads and no cache would hold until the next call pass it by
    // (LayerParams::once)
    auto load_inside = [&](auto once, Chunk &c, int ch) {
        typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
        const int64_t k0 = (int64_t)ch * KC;
        if constexpr (BT) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const uint8_t *from = B + E * k0 + (brow[i] + 16u * lq);
                if constexpr (once.value) c.b[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4u *>(from));
                else c.b[i] = ldg16(from);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NB; ++i) c.b[i] = ldg16(B + (k0 + RPL * i) * p.ldb * E + brow[0]);
        }
#pragma unroll
        for (int i = 0; i < NA; ++i) c.a[i] = ldg16(A + E * k0 + (arow[i] + 16u * lq));
    };
    // a chunk that crosses the end of K: zeros past it
    auto load_end = [&](Chunk &c, int ch) {
        const int k0 = ch * KC;
        if constexpr (BT) {
#pragma unroll
            for (int i = 0; i < NB; ++i) c.b[i] = row_end<E>(B + brow[i], k0 + VE * lq, p.K);
        } else {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int k = k0 + RPL * i + br;
                c.b[i] = row_end<E>(B + (int64_t)min(k, p.K - 1) * p.ldb * E, bc, p.N);
                if (k >= p.K) c.b[i] = u32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < NA; ++i) c.a[i] = row_end<E>(A + arow[i], k0 + VE * lq, p.K);
    };

    // B stored K x N in the slot: row r keeps 16-byte piece q at q ^ sw(r).  16 bits: the transposing read's
    // lane a of each 16 takes row a / 4 + 8 g (and + 4), columns 4 (a % 4) .. +3, and two groups g are served
    // together; fp32: the groups take rows 4 apart.  Their rows' pieces stand in different banks.
    auto sw = [](int r) {
        if constexpr (E == 4) return CG == 4 ? ((r >> 2) & 3) << 2 : ((r >> 2) & 1) << 2;
        else return CG == 4 ? (((r >> 1) & 1) << 1) | (((r >> 3) & 1) << 2) : ((r >> 3) & 1) << 1;
    };
    const int rb = 8 * g + ((lane & 15) >> 2);

    f32x4 acc[RT][CG];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < CG; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
    auto stage = [&](const Chunk &c) {
        staging_order();                                     // the last chunk's reads come first
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = BT ? piece<KB>(RPI * i + lr, lq) : 1024 * i + br * 16 * LPR + ((bq ^ sw(RPL * i + br)) << 4);
            *reinterpret_cast<u32x4 *>(slot + at) = c.b[i];
        }
#pragma unroll
        for (int i = 0; i < NA; ++i) *reinterpret_cast<u32x4 *>(slot + OFF_A + piece<KB>(RPI * i + lr, lq)) = c.a[i];
        staging_order();
    };
    auto compute = [&]() {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            u32x4 a[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) a[r] = *reinterpret_cast<const u32x4 *>(slot + OFF_A + piece<KB>(16 * r + (lane & 15), 4 * i + g));
#pragma unroll
            for (int j = 0; j < CG; ++j) {
                u32x4 b;
                if constexpr (BT) {
                    b = *reinterpret_cast<const u32x4 *>(slot + piece<KB>(16 * j + (lane & 15), 4 * i + g));
                } else if constexpr (E == 2) {
                    const uint8_t *q = slot + (32 * i + rb) * 16 * LPR + (((2 * j + ((lane & 3) >> 1)) ^ sw(rb)) << 4) + (lane & 1) * 8;
                    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)q);
                    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(q + 4 * 16 * LPR));
                    b = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int k = 16 * i + 4 * g + e;
                        b[e] = *reinterpret_cast<const uint32_t *>(slot + k * 16 * LPR + (((4 * j + ((lane & 15) >> 2)) ^ sw(k)) << 4) + (lane & 3) * 4);
                    }
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) acc[r][j] = TI::mma16(a[r], b, acc[r][j]);
            }
        }
    };

    // Column tiles start at different chunks: in step, all of the chip would ask for the same piece of every
    // row.  The chunks that need care (at most two) come last, one by one.
    const int n = max(min(c1, last >= 0 ? last / KC + 1 : 0) - c0, 0);
    const int turn = n > 0 ? tn % n : 0;
    auto at = [&](int i) {
        const int c = i + turn;
        return c0 + (c < n ? c : c - n);
    };
    Chunk x[DEPTH];
    auto walk = [&](auto once) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (d < n) load_inside(once, x[d], at(d));
        int i = 0;
#pragma unroll 1
        for (; i + 2 * DEPTH <= n; i += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                stage(x[d]);
                load_inside(once, x[d], at(i + d + DEPTH));
                compute();
            }
        }
#pragma unroll 1
        for (; i < n; i += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
                if (i + d < n) {
                    stage(x[d]);
                    if (i + d + DEPTH < n) load_inside(once, x[d], at(i + d + DEPTH));
                    compute();
                }
        }
    };
    if constexpr (BT) {
        if (p.once) walk(std::true_type());
        else walk(std::false_type());
    } else {
        walk(std::false_type());
    }
#pragma unroll 1
    for (int c = c0 + n; c < c1; ++c) {
        load_end(x[0], c);
        stage(x[0]);
        compute();
    }

    __syncthreads();                                         // the slots become the sums
    f32x4 *part = reinterpret_cast<f32x4 *>(smem);           // [wave][r][j][lane]
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < CG; ++j) part[((wave * RT + r) * CG + j) * 64 + lane] = acc[r][j];
    __syncthreads();
    // wave w finishes tiles w, w + 8, ...: lane holds rows 4 * (lane / 16) + e of one column
    const T *X = static_cast<const T *>(p.grad ? p.Z : p.C);
    T *D = static_cast<T *>(p.D), *Z = p.grad ? nullptr : static_cast<T *>(p.Z);
#pragma unroll 1
    for (int t = wave; t < RT * CG; t += WAVES) {
        f32x4 sum = part[t * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += part[(w * RT * CG + t) * 64 + lane];
        const int n = n0 + 16 * (t % CG) + (lane & 15), m0 = 16 * (t / CG) + 4 * g;
        if (n >= p.N || m0 >= p.M) continue;
        const float bias = p.has_bias ? static_cast<const float *>(p.bias)[n] : 0.0f;
        // rows past the range take its last one's values; they are not stored
        float v[4];
        T xv[4], out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = __builtin_fmaf(p.alpha, sum[e], bias);
            xv[e] = p.grad || p.has_beta ? X[(int64_t)min(m0 + e, p.M - 1) * p.ldc + n] : (T)0;
        }
        if (Z) {
            round_values(v, out);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m0 + e < p.M) Z[(int64_t)(m0 + e) * p.ldc + n] = out[e];
        }
        finish_values<4, (int)sizeof(T)>(p, v, xv);
        round_values(v, out);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (m0 + e < p.M) D[(int64_t)(m0 + e) * p.ldc + n] = out[e];
    }
}

template <class TI, class TO, bool BT, int RT, int CG, int KB>
hipError_t launch(const LayerParams &p, unsigned grid, hipStream_t s) {
    hipLaunchKernelGGL((layer_rows<TI, TO, BT, RT, CG, KB>), dim3(grid), dim3(WAVES * 64), 0, s, p);
    return hipGetLastError();
}

template <class TI, class TO>
const LayerEntry *lookup(int op_b, int rt, int cg) {
    // [rt 1, 2, 4][narrow, wide]
    static const LayerEntry n[3][2] = {{{launch<TI, TO, false, 1, 2, 128>, 16, 32, "layer_rows_16x32"},
                                        {launch<TI, TO, false, 1, 4, 128>, 16, 64, "layer_rows_16x64"}},
                                       {{launch<TI, TO, false, 2, 2, 128>, 32, 32, "layer_rows_32x32"},
                                        {launch<TI, TO, false, 2, 4, 128>, 32, 64, "layer_rows_32x64"}},
                                       {{launch<TI, TO, false, 4, 2, 128>, 64, 32, "layer_rows_64x32"},
                                        {launch<TI, TO, false, 4, 4, 128>, 64, 64, "layer_rows_64x64"}}};
    static const LayerEntry t[3][2] = {{{launch<TI, TO, true, 1, 1, 256>, 16, 16, "layer_rows_16x16"},
                                        {launch<TI, TO, true, 1, 4, 128>, 16, 64, "layer_rows_16x64"}},
                                       {{launch<TI, TO, true, 2, 1, 256>, 32, 16, "layer_rows_32x16"},
                                        {launch<TI, TO, true, 2, 4, 128>, 32, 64, "layer_rows_32x64"}},
                                       {{launch<TI, TO, true, 4, 1, 256>, 64, 16, "layer_rows_64x16"},
                                        {launch<TI, TO, true, 4, 4, 128>, 64, 64, "layer_rows_64x64"}}};
    if (op_b < 0 || op_b > 1 || (rt != 1 && rt != 2 && rt != 4) || (cg != 4 && cg != (op_b ? 1 : 2))) return nullptr;
    return &(op_b ? t : n)[rt >> 1][cg == 4];
}

}  // namespace

#if defined(TGE_PAIR_F32_F32)
const LayerEntry *layer_rows_f32_f32(int b, int rt, int cg) { return lookup<TF32, OF32>(b, rt, cg); }
#elif defined(TGE_PAIR_F16_F16)
const LayerEntry *layer_rows_f16_f16(int b, int rt, int cg) { return lookup<TF16, OF16>(b, rt, cg); }
#elif defined(TGE_PAIR_F16_F32)
const LayerEntry *layer_rows_f16_f32(int b, int rt, int cg) { return lookup<TF16, OF32>(b, rt, cg); }
#elif defined(TGE_PAIR_BF16_BF16)
const LayerEntry *layer_rows_bf16_bf16(int b, int rt, int cg) { return lookup<TBF16, OBF16>(b, rt, cg); }
#elif defined(TGE_PAIR_BF16_F32)
const LayerEntry *layer_rows_bf16_f32(int b, int rt, int cg) { return lookup<TBF16, OF32>(b, rt, cg); }
#else
#error "define one TGE_PAIR_* macro of a float type"
#endif

}  // namespace tge
