// Products of few rows per expert on gfx950, any alignment and any K: 16 rows and 16 * CG columns
// of one expert per workgroup.  Bound by the weights' bytes, each read once (twice 16 rows read
// them twice, mostly from cache): 64 rows over 64 experts of 2048 x 4096 (bf16, B transposed; 38 have
// rows) 109 us, 5.7 TB/s.  Few or small experts are bound by the launch (2.9 us) and the latency of a
// wave's chunks, one after another: 8 rows over 16 experts of 1024 x 2048 7.2 us (cold 8.6).
//
// K is divided over the 8 waves of a workgroup (4 and 16 measured no better): with few rows a
// workgroup per tile walks K too slowly (9 rows over 2 experts of 2745 x 6793: 93 us in 128-wide
// tiles, 22 us here).  Each wave takes its part in chunks of KC k, one chunk in registers in flight
// while the one before is multiplied; a private LDS slot only changes the lane order:
//
//  * an operand whose rows lie along K (A, a transposed B) is loaded 4 lanes per row (whole
//    64-byte pieces) and read as fragments, row lane % 16, 8 k of piece lane / 16;
//  * a B stored K x N is loaded 8 lanes per row of 64 columns (4 per row of 32: a workgroup streams
//    some 60 GB/s, so few columns take narrower workgroups) and read with the transposing read
//    ds_read_b64_tr_b16 (the lane map of gemm_skinny.hip).
//
// The direct-to-LDS loads of gemm_skinny.hip need 16-byte alignment and a whole number of 64-byte
// pieces in K; ordinary loads do not.  Loads that would cross the end of K are moved back and their
// values down (ldg16_row_end); a column tile that reaches past N starts its loads at the row's last
// element at most and reads on into the next row, which gives columns that are never stored.
//
// Preconditions (checked by the host): 16-bit types, K >= 8, N >= 8 when B is not transposed.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"

namespace tge {
namespace {

using namespace dev;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int WAVES = 8;

// 16 rows x 64 bytes: 16-byte piece q of row r, at q ^ {0, 2, 3, 1}[r / 4] (a 16-byte read serves lanes
// 0-3, 12-15, 20-23 and 24-27 together, then 4-11, 16-19 and 28-31: 16 different places either way)
__device__ __forceinline__ int piece16(int r, int q) {
    const int t = r >> 2;
    return r * 64 + ((q ^ ((t << 1) & 2) ^ (t & 2 ? 3 : 0)) << 4);
}

// Orders this wave's LDS accesses (they execute in order; no instruction).
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// BT: B stored N x K; CG: groups of 16 columns; KC: k per chunk.
template <class TI, class TO, bool BT, int CG, int KC>
__global__ __launch_bounds__(WAVES * 64, 2) void gemm_rows16(GroupedParams p) {
    using T = typename TO::T;
    static_assert(BT || ((CG == 4 || CG == 2) && KC == 64), "rows of 64 or 32 columns");
    constexpr int NI = KC / 32;                              // 16x16x32 instructions per chunk and group
    constexpr int LPR = 2 * CG, RPL = 64 / LPR;              // K x N: lanes per row, rows per load
    constexpr int NL = BT ? CG * NI : KC / RPL;              // 1 KiB loads of B per chunk
    constexpr int COLS = 16 * CG;
    constexpr int OFF_A = NL * 1024, SLOT = OFF_A + NI * 1024;
    static_assert(SLOT >= CG * 1024, "the slots hold the waves' sums at the end");
    __shared__ __attribute__((aligned(16))) uint8_t smem[WAVES * SLOT];

    int tn;
    if (!select_rows<2, (int)sizeof(T)>(p, blockIdx.x, 16, tn)) return;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane >> 2, lq = lane & 3;                 // load order of rows along K: row, piece
    const int n0 = tn * COLS;
    const int nch = (p.K + KC - 1) / KC;
    const int c0 = (int)((int64_t)nch * wave / WAVES), c1 = (int)((int64_t)nch * (wave + 1) / WAVES);
    uint8_t *const slot = smem + wave * SLOT;
    const int put = piece16(lr, lq), get = piece16(lane & 15, g);

    const uint8_t *arow = static_cast<const uint8_t *>(p.A) + (int64_t)min(lr, p.M - 1) * p.lda * 2 + 16 * lq;
    // BT: row n0 + 16 j + lr of B.  Else: row lane / LPR of the load, 8 columns from n0 + 8 * (lane % LPR)
    const uint8_t *brow[BT ? CG : 1];
    const int br = lane / LPR, bq = lane % LPR, bc = n0 + 8 * bq, bcol = min(bc, p.N - 1);
    if constexpr (BT) {
#pragma unroll
        for (int j = 0; j < CG; ++j)
            brow[j] = static_cast<const uint8_t *>(p.B) + (int64_t)min(n0 + 16 * j + lr, p.N - 1) * p.ldb * 2 + 16 * lq;
    } else {
        brow[0] = static_cast<const uint8_t *>(p.B) + ((int64_t)br * p.ldb + bcol) * 2;
    }
    // (uniform) a chunk whose loads need no care: inside K; with columns past N also a row after it
    const int last = p.K - KC - (!BT && n0 + COLS > p.N ? 1 : 0);

    struct Chunk {
        u32x4 b[NL], a[NI];
    };
    auto load = [&](Chunk &c, int ch) {
        const int k0 = ch * KC;
        if (k0 <= last) {
            if constexpr (BT) {
#pragma unroll
                for (int j = 0; j < CG; ++j)
#pragma unroll
                    for (int i = 0; i < NI; ++i) c.b[j * NI + i] = ldg16(brow[j] + 2 * (k0 + 32 * i));
            } else {
#pragma unroll
                for (int i = 0; i < NL; ++i) c.b[i] = ldg16(brow[0] + (int64_t)(k0 + RPL * i) * p.ldb * 2);
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) c.a[i] = ldg16(arow + 2 * (k0 + 32 * i));
        } else {   // zeros past K
            if constexpr (BT) {
#pragma unroll
                for (int j = 0; j < CG; ++j)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        c.b[j * NI + i] = ldg16_row_end(brow[j] - 16 * lq, k0 + 32 * i + 8 * lq, p.K);
            } else {
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const int k = k0 + RPL * i + br;
                    c.b[i] = ldg16_row_end(static_cast<const uint8_t *>(p.B) + (int64_t)min(k, p.K - 1) * p.ldb * 2, bc, p.N);
                    if (k >= p.K) c.b[i] = u32x4{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i)
                c.a[i] = ldg16_row_end(arow - 16 * lq, k0 + 32 * i + 8 * lq, p.K);
        }
    };

    // B stored K x N in the slot: row r of 128 (64) bytes keeps 16-byte piece q at q ^ sw(r); the
    // transposing read's lane a of each 16 takes row a / 4 + 8 g (and + 4), columns 4 (a % 4) .. +3,
    // and two groups g are served together: their rows' pieces stand in different banks
    auto sw = [](int r) { return CG == 4 ? (((r >> 1) & 1) << 1) | (((r >> 3) & 1) << 2) : ((r >> 3) & 1) << 1; };
    const int rb = 8 * g + ((lane & 15) >> 2);

    f32x4 acc[CG];
#pragma unroll
    for (int j = 0; j < CG; ++j) acc[j] = f32x4{0, 0, 0, 0};
    auto stage = [&](const Chunk &c) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int at = BT ? put : br * 16 * LPR + ((bq ^ sw(RPL * i + br)) << 4);
            *reinterpret_cast<u32x4 *>(slot + 1024 * i + at) = c.b[i];
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) *reinterpret_cast<u32x4 *>(slot + OFF_A + 1024 * i + put) = c.a[i];
    };
    auto compute = [&]() {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(slot + OFF_A + 1024 * i + get);
#pragma unroll
            for (int j = 0; j < CG; ++j) {
                u32x4 b;
                if constexpr (BT) {
                    b = *reinterpret_cast<const u32x4 *>(slot + 1024 * (j * NI + i) + get);
                } else {
                    const uint8_t *q = slot + (32 * i + rb) * 16 * LPR + (((2 * j + ((lane & 3) >> 1)) ^ sw(rb)) << 4) + (lane & 1) * 8;
                    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)q);
                    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(q + 4 * 16 * LPR));
                    b = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
                acc[j] = TI::mma16(a, b, acc[j]);
            }
        }
    };

    if (c0 < c1) {
        Chunk x;
        load(x, c0);
#pragma unroll 1
        for (int ch = c0; ch < c1; ++ch) {
            wave_order();                                    // the last chunk's reads come first
            stage(x);
            wave_order();
            if (ch + 1 < c1) load(x, ch + 1);                // in flight while this chunk is multiplied
            compute();
        }
    }

    __syncthreads();                                         // the slots become the sums
    f32x4 *part = reinterpret_cast<f32x4 *>(smem);           // [wave][j][lane]
#pragma unroll
    for (int j = 0; j < CG; ++j) part[(wave * CG + j) * 64 + lane] = acc[j];
    __syncthreads();
    // wave j finishes column group j: lane holds rows 4 * (lane / 16) + r of one column
    if (wave >= CG) return;
    f32x4 sum = part[wave * 64 + lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += part[(w * CG + wave) * 64 + lane];
    const int n = n0 + 16 * wave + (lane & 15);
    if (n >= p.N) return;
    const float bias = p.has_bias ? static_cast<const float *>(p.bias)[n] : 0.0f;
    const T *C = static_cast<const T *>(p.C);
    T *D = static_cast<T *>(p.D);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int m = 4 * g + r;
        if (m >= p.M) continue;
        const int64_t idx = (int64_t)m * p.ldc + n;
        float x = p.alpha * sum[r];
        if (p.gate) x = (float)C[idx] > 0.0f ? x : 0.0f;
        else if (p.has_beta) x += p.beta * (float)C[idx];
        x += bias;
        if (p.relu) x = x > 0.0f ? x : 0.0f;
        D[idx] = (T)x;
    }
}

template <class TI, class TO, bool BT, int CG, int KC>
hipError_t launch(const GroupedParams &p, unsigned grid, hipStream_t s) {
    hipLaunchKernelGGL((gemm_rows16<TI, TO, BT, CG, KC>), dim3(grid), dim3(WAVES * 64), 0, s, p);
    return hipGetLastError();
}

template <class TI, class TO>
const GroupedEntry *lookup(int op_b, int cg) {
    static const GroupedEntry n[2] = {{launch<TI, TO, false, 2, 64>, 16, 32, "gemm_rows16_16x32"},
                                      {launch<TI, TO, false, 4, 64>, 16, 64, "gemm_rows16_16x64"}};
    static const GroupedEntry t[2] = {{launch<TI, TO, true, 1, 128>, 16, 16, "gemm_rows16_16x16"},
                                      {launch<TI, TO, true, 4, 64>, 16, 64, "gemm_rows16_16x64"}};
    if (op_b == 0) return cg == 2 ? &n[0] : cg == 4 ? &n[1] : nullptr;
    return op_b == 1 ? (cg == 1 ? &t[0] : cg == 4 ? &t[1] : nullptr) : nullptr;
}

}  // namespace

#if defined(TGE_PAIR_F16_F16)
const GroupedEntry *grouped_rows16_f16_f16(int b, int cg) { return lookup<TF16, OF16>(b, cg); }
#elif defined(TGE_PAIR_F16_F32)
const GroupedEntry *grouped_rows16_f16_f32(int b, int cg) { return lookup<TF16, OF32>(b, cg); }
#elif defined(TGE_PAIR_BF16_BF16)
const GroupedEntry *grouped_rows16_bf16_bf16(int b, int cg) { return lookup<TBF16, OBF16>(b, cg); }
#elif defined(TGE_PAIR_BF16_F32)
const GroupedEntry *grouped_rows16_bf16_f32(int b, int cg) { return lookup<TBF16, OF32>(b, cg); }
#else
#error "define one TGE_PAIR_* macro of a 16-bit float type"
#endif

}  // namespace tge
