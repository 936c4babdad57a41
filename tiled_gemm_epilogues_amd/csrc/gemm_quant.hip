// Products with 4-bit weights on gfx950: D = act(alpha * A * W^T + beta * C + bias), where row n of
// W holds K codes q of 4 bits and, per block of G consecutive k, a scale s and a zero point z:
//
//   W[n][k] = s[n][k / G] * (q[n][k] - z[n][k / G])
//   D[m][n] = sum over blocks b of  s[n][b] * ( sum over k in b of  A[m][k] * (q[n][k] - z[n][b]) )
//
// The inner sums run on the matrix cores in the type of A, in which the small integers are exact,
// and the scale multiplies each block's sum in fp32: no weight is ever rounded.
//
// Codes become 16-bit floats by bit operations: the 4 bits are moved to the upper mantissa bits
// below the exponent of 16.0, which gives 16 + q.  One 32-bit word of 8 codes yields the pairs
// (k, k+4), k = 0 .. 3, with one shift and one and-or each; A's 8 values of the same k are brought
// into that order with four byte permutes.  For fp16 the offset 16 + z is subtracted with packed
// adds (exact).  bf16 has no packed add, so its sums keep the offset,
//
//   sum A * (q - z) = sum A * (16 + q) - (16 + z) * sum A,
//
// with sum A from one more matrix instruction per A fragment, against a fragment of ones.  The
// terms are at most 31 / 8 times larger than a centred sum's: two bits of fp32's 24.
//
// A lane of a 16x16x32 matrix instruction holds 8 k of one weight row (n = lane % 16).  A 16-byte
// load of a lane covers 32 k of its row: lanes g = lane / 16 hold k = 32g .. 32g+31 of a chunk of
// 128.  With G >= 128 the chunk's four instructions may take any 8 of each lane.  With G = 64 and
// 32 an instruction must stay inside one block: the four words are exchanged between the lane
// groups (permlane32_swap, then permlane16_swap) so that word i belongs to block i / 2, or i.
// kofs() is the resulting k of word i in lane group g; A is loaded to match.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"

namespace tge {
namespace {

using namespace dev;

constexpr int CHUNK = 128;    // k per step: 16 bytes of codes per lane

// first of the 8 k (within a chunk) of word i in lane group g
template <int G>
__device__ __forceinline__ int kofs(int i, int g) {
    if constexpr (G >= 128) return 32 * g + 8 * i;
    else if constexpr (G == 64) return 64 * (i >> 1) + 32 * (g & 1) + 16 * (g >> 1) + 8 * (i & 1);
    else return 32 * i + 8 * g;
}

// the four words of a lane's 16 code bytes, exchanged between the lane groups (see above)
template <int G>
__device__ __forceinline__ u32x4 exchange(u32x4 w) {
    if constexpr (G <= 64) {
        const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
        w = u32x4{a[0], b[0], a[1], b[1]};
    }
    if constexpr (G <= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
        const auto b = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
        w = u32x4{a[0], a[1], b[0], b[1]};
    }
    return w;
}

// 8 values of A in the order of the code pairs: (0,4) (1,5) (2,6) (3,7)
__device__ __forceinline__ u32x4 pair_order(u32x4 a) {
    return u32x4{__builtin_amdgcn_perm(a[2], a[0], 0x05040100u), __builtin_amdgcn_perm(a[2], a[0], 0x07060302u),
                 __builtin_amdgcn_perm(a[3], a[1], 0x05040100u), __builtin_amdgcn_perm(a[3], a[1], 0x07060302u)};
}

// 16 + q of the 8 codes of a word, as pairs (0,4) (1,5) (2,6) (3,7)
template <class TI>
__device__ __forceinline__ u32x4 codes16(uint32_t w);
template <>
__device__ __forceinline__ u32x4 codes16<TF16>(uint32_t w) {
    constexpr uint32_t m = 0x03c003c0u, o = 0x4c004c00u;   // mantissa bits 6-9; 16.0
    return u32x4{((w << 6) & m) | o, ((w << 2) & m) | o, ((w >> 2) & m) | o, ((w >> 6) & m) | o};
}
template <>
__device__ __forceinline__ u32x4 codes16<TBF16>(uint32_t w) {
    constexpr uint32_t m = 0x00780078u, o = 0x41804180u;   // mantissa bits 3-6; 16.0
    return u32x4{((w << 3) & m) | o, ((w >> 1) & m) | o, ((w >> 5) & m) | o, ((w >> 9) & m) | o};
}

typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// What one lane's weight row contributes to a block: scale, and the offset 16 + z to take off.
template <class TI>
struct Block {
    float s;
    float off;               // 16 + z
};

template <class TI>
struct Quant;
template <>
struct Quant<TF16> {
    using T = _Float16;
    static constexpr bool SUMS = false;
    // q - z of a word's codes (exact: integers below 32 in magnitude)
    __device__ static u32x4 values(uint32_t w, float off) {
        u32x4 v = codes16<TF16>(w);
        const _Float16 o = (_Float16)off;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = v[i];
            v[i] = __builtin_bit_cast(uint32_t, (h2)(__builtin_bit_cast(h2, x) - (h2){o, o}));
        }
        return v;
    }
    __device__ static constexpr uint32_t ones() { return 0x3c003c00u; }
};
template <>
struct Quant<TBF16> {
    using T = __bf16;
    static constexpr bool SUMS = true;
    __device__ static u32x4 values(uint32_t w, float) { return codes16<TBF16>(w); }
    __device__ static constexpr uint32_t ones() { return 0x3f803f80u; }
};

// Scale and offset of block b of the weight row whose blocks start at `row`; a chunk's blocks past
// K get the last block's offset and a zero scale (A is zero there).
template <class TI>
__device__ __forceinline__ Block<TI> block_of(const QuantParams &p, int64_t row, int b, int nblk) {
    const int64_t i = row + min(b, nblk - 1);
    Block<TI> x;
    x.s = b < nblk ? (float)static_cast<const typename Quant<TI>::T *>(p.scales)[i] : 0.0f;
    x.off = 16.0f + (p.zeros ? (float)p.zeros[i] : 8.0f);
    return x;
}

// The expert, row tile and column tile of a workgroup; false: none.  With one weight matrix the
// tiles of one row tile are consecutive in columns; A, C, D and p.M are moved to the row tile.
template <int ECD>
__device__ __forceinline__ bool select_tile(QuantParams &p, int bm, int &tn) {
    if (p.offs) {
        int e = 0;
        if (!select_rows<2, ECD>(p, blockIdx.x, bm, tn, &e)) return false;
        p.Q += e * p.stride_q;
        p.scales = static_cast<const uint8_t *>(p.scales) + e * p.stride_s * 2;
        if (p.zeros) p.zeros += e * p.stride_s;
        return true;
    }
    int tm;
    raster(xcd_remap(blockIdx.x, gridDim.x), p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int64_t row = (int64_t)tm * bm;
    p.M -= (int)row;
    p.A = static_cast<const uint8_t *>(p.A) + row * p.lda * 2;
    if (p.C) p.C = static_cast<const uint8_t *>(p.C) + row * p.ldc * ECD;
    p.D = static_cast<uint8_t *>(p.D) + row * p.ldc * ECD;
    return true;
}

// One output element: the epilogue on its sum.
template <class T>
__device__ __forceinline__ void store_one(const QuantParams &p, int m, int n, float sum, float bias) {
    const int64_t idx = (int64_t)m * p.ldc + n;
    float x = p.alpha * sum;
    if (p.has_beta) x += p.beta * (float)static_cast<const T *>(p.C)[idx];
    x += bias;
    if (p.relu) x = x > 0.0f ? x : 0.0f;
    static_cast<T *>(p.D)[idx] = (T)x;
}

// ---- few rows ----------------------------------------------------------------------------------
// 16 * MT rows and 16 columns per workgroup: the weights are read once, straight into registers
// (they are used once: LDS would only add a trip), by WAVES waves that take every WAVES-th chunk
// of K, so that a workgroup reads whole lines of its 16 weight rows and enough loads are in
// flight; DEPTH chunks per wave are loaded ahead.  A comes from L2 (every workgroup reads it).
// The waves' sums are added through LDS in wave order.
constexpr int WAVES = 8;
constexpr int NB = 16;

template <class TI, int G, int MT>
struct RowsChunk {
    static constexpr int NBLK = G >= 128 ? 1 : CHUNK / G;    // blocks per chunk
    u32x4 q;
    u32x4 a[MT][4];
    Block<TI> blk[NBLK];
};

template <class TI, class TO, int G, int MT>
__global__ __launch_bounds__(WAVES * 64) void quant_rows(QuantParams p) {
    using T = typename TO::T;
    using QT = Quant<TI>;
    using CH = RowsChunk<TI, G, MT>;
    constexpr int DEPTH = MT == 1 ? 4 : 2;
    constexpr int SUB = G >= 128 ? 4 : G / 32;               // matrix instructions per block
    __shared__ f32x4 part[WAVES][MT][64];

    int tn;
    if (!select_tile<(int)sizeof(T)>(p, 16 * MT, tn)) return;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = tn * NB + (lane & 15), nc = min(n, p.N - 1);
    const uint8_t *qrow = p.Q + (int64_t)nc * p.ldq + 16 * g;
    const int64_t srow = (int64_t)nc * p.lds;
    const uint8_t *arow[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
        arow[t] = static_cast<const uint8_t *>(p.A) + (int64_t)min(16 * t + (lane & 15), p.M - 1) * p.lda * 2;
    const int nch = (p.K + CHUNK - 1) / CHUNK, nblk = p.K / p.block;

    auto load = [&](CH &c, int ch) {
        const int k0 = ch * CHUNK;
        // the last chunk may end inside (whole blocks of 32): zeros there
        c.q = u32x4{0, 0, 0, 0};
        if (k0 + 32 * g < p.K) c.q = ldg16(qrow + k0 / 2);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = k0 + kofs<G>(i, g);
                c.a[t][i] = u32x4{0, 0, 0, 0};
                if (k < p.K) c.a[t][i] = ldg16(arow[t] + 2 * k);
            }
        const int b0 = G >= 128 ? k0 / p.block : k0 / G;
#pragma unroll
        for (int b = 0; b < CH::NBLK; ++b) c.blk[b] = block_of<TI>(p, srow, b0 + b, nblk);
    };

    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    auto compute = [&](const CH &c) {
        const u32x4 w = exchange<G>(c.q);
        const u32x4 one = u32x4{QT::ones(), QT::ones(), QT::ones(), QT::ones()};
#pragma unroll
        for (int b = 0; b < CH::NBLK; ++b) {
            f32x4 t[MT], sum[MT];
#pragma unroll
            for (int r = 0; r < MT; ++r) t[r] = sum[r] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = b * SUB; i < (b + 1) * SUB; ++i) {
                const u32x4 v = QT::values(w[i], c.blk[b].off);
#pragma unroll
                for (int r = 0; r < MT; ++r) {
                    const u32x4 a = pair_order(c.a[r][i]);
                    t[r] = TI::mma16(a, v, t[r]);
                    if constexpr (QT::SUMS) sum[r] = TI::mma16(a, one, sum[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < MT; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = QT::SUMS ? __builtin_fmaf(-c.blk[b].off, sum[r][e], t[r][e]) : t[r][e];
                    acc[r][e] = __builtin_fmaf(c.blk[b].s, x, acc[r][e]);
                }
        }
    };

    CH buf[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (wave + d * WAVES < nch) load(buf[d], wave + d * WAVES);
    for (int c0 = wave; c0 < nch; c0 += DEPTH * WAVES) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int c = c0 + d * WAVES;
            if (c < nch) {
                compute(buf[d]);
                if (c + DEPTH * WAVES < nch) load(buf[d], c + DEPTH * WAVES);
            }
        }
    }

#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave >= MT) return;
    // wave t finishes row tile t: lane holds rows 4 * (lane / 16) + r of column n
    f32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += part[w][wave][lane];
    if (n >= p.N) return;
    const float bias = p.has_bias ? static_cast<const float *>(p.bias)[n] : 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int m = 16 * wave + 4 * g + r;
        if (m < p.M) store_one<T>(p, m, n, sum[r], bias);
    }
}

// ---- many rows ---------------------------------------------------------------------------------
// 128 x 128 output tile, 4 waves of 64 x 64.  A is staged in LDS once per workgroup, already in
// pair order (global -> registers -> permute -> LDS, two stages of 128 k, rows of 256 bytes whose
// 16-byte piece c stands at c ^ (row % 16)); each wave turns the codes of its 64 columns into
// fragments in registers, straight from global memory one chunk ahead.
constexpr int TM = 128, TN = 128, TNT = 256;

template <class TI, class TO, int G>
__global__ __launch_bounds__(TNT, 2) void quant_tile(QuantParams p) {
    using T = typename TO::T;
    using QT = Quant<TI>;
    constexpr int NBLK = G >= 128 ? 1 : CHUNK / G;
    constexpr int SUB = G >= 128 ? 4 : G / 32;
    constexpr int STAGE = TM * CHUNK * 2;
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * STAGE];

    int tn;
    if (!select_tile<(int)sizeof(T)>(p, TM, tn)) return;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int nch = (p.K + CHUNK - 1) / CHUNK, nblk = p.K / p.block;

    // staging: thread -> piece tid % 16 of rows tid / 16 + 16 i
    const uint8_t *asrc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asrc[i] = static_cast<const uint8_t *>(p.A) + (int64_t)min((tid >> 4) + 16 * i, p.M - 1) * p.lda * 2 + (tid & 15) * 16;
    u32x4 st[8];
    auto fetch = [&](int ch) {
        const bool in = ch * CHUNK + (tid & 15) * 8 < p.K;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            st[i] = u32x4{0, 0, 0, 0};
            if (in) st[i] = ldg16(asrc[i] + ch * CHUNK * 2);
        }
    };
    auto put = [&](int stage) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = (tid >> 4) + 16 * i;
            *reinterpret_cast<u32x4 *>(smem + stage * STAGE + row * 256 + (((tid & 15) ^ (row & 15)) << 4)) = pair_order(st[i]);
        }
    };
    // weights: column group j of the wave
    const uint8_t *qrow[4];
    int64_t srow[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = min(tn * TN + wn * 64 + 16 * j + (lane & 15), p.N - 1);
        qrow[j] = p.Q + (int64_t)n * p.ldq + 16 * g;
        srow[j] = (int64_t)n * p.lds;
    }
    u32x4 q[4];
    Block<TI> blk[4][NBLK];
    auto weights = [&](int ch) {
        const int k0 = ch * CHUNK;
        const int b0 = G >= 128 ? k0 / p.block : k0 / G;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            q[j] = u32x4{0, 0, 0, 0};
            if (k0 + 32 * g < p.K) q[j] = ldg16(qrow[j] + k0 / 2);
#pragma unroll
            for (int b = 0; b < NBLK; ++b) blk[j][b] = block_of<TI>(p, srow[j], b0 + b, nblk);
        }
    };

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    if (nch > 0) {
        fetch(0);
        weights(0);
        put(0);
    }
    __syncthreads();
    const u32x4 one = u32x4{QT::ones(), QT::ones(), QT::ones(), QT::ones()};
    for (int ch = 0; ch < nch; ++ch) {
        const bool more = ch + 1 < nch;
        u32x4 w[4];
        Block<TI> bl[4][NBLK];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] = exchange<G>(q[j]);
#pragma unroll
            for (int b = 0; b < NBLK; ++b) bl[j][b] = blk[j][b];
        }
        if (more) {
            fetch(ch + 1);
            weights(ch + 1);
        }
        const uint8_t *la = smem + (ch & 1) * STAGE + (wm * 64 + (lane & 15)) * 256;
#pragma unroll
        for (int b = 0; b < NBLK; ++b) {
            f32x4 t[4][4], sum[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[i] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 4; ++j) t[i][j] = f32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int s = b * SUB; s < (b + 1) * SUB; ++s) {
                u32x4 a[4];
                const int piece = kofs<G>(s, g) / 8;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[i] = *reinterpret_cast<const u32x4 *>(la + i * 16 * 256 + ((piece ^ (lane & 15)) << 4));
                if constexpr (QT::SUMS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] = TI::mma16(a[i], one, sum[i]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x4 v = QT::values(w[j][s], bl[j][b].off);
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[i][j] = TI::mma16(a[i], v, t[i][j]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = QT::SUMS ? __builtin_fmaf(-bl[j][b].off, sum[i][e], t[i][j][e]) : t[i][j][e];
                        acc[i][j][e] = __builtin_fmaf(bl[j][b].s, x, acc[i][j][e]);
                    }
        }
        if (more) put((ch + 1) & 1);
        __syncthreads();
    }

#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = tn * TN + wn * 64 + 16 * j + (lane & 15);
        if (n >= p.N) continue;
        const float bias = p.has_bias ? static_cast<const float *>(p.bias)[n] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = wm * 64 + 16 * i + 4 * g + r;
                if (m < p.M) store_one<T>(p, m, n, acc[i][j][r], bias);
            }
    }
}

// ---- entries -----------------------------------------------------------------------------------

template <class TI, class TO, int G, int MT>
hipError_t launch_rows(const QuantParams &p, unsigned grid, hipStream_t s) {
    hipLaunchKernelGGL((quant_rows<TI, TO, G, MT>), dim3(grid), dim3(WAVES * 64), 0, s, p);
    return hipGetLastError();
}
template <class TI, class TO, int G>
hipError_t launch_tile(const QuantParams &p, unsigned grid, hipStream_t s) {
    hipLaunchKernelGGL((quant_tile<TI, TO, G>), dim3(grid), dim3(TNT), 0, s, p);
    return hipGetLastError();
}

template <class TI, class TO, int G>
const QuantEntry *rows_entry(int mt) {
    static const QuantEntry e[3] = {{launch_rows<TI, TO, G, 1>, 16, NB, "quant_rows_m16"},
                                    {launch_rows<TI, TO, G, 2>, 32, NB, "quant_rows_m32"},
                                    {launch_rows<TI, TO, G, 4>, 64, NB, "quant_rows_m64"}};
    return mt == 1 ? &e[0] : mt == 2 ? &e[1] : mt == 4 ? &e[2] : nullptr;
}
template <class TI, class TO>
const QuantEntry *lookup_rows(int block, int mt) {
    return block == 32 ? rows_entry<TI, TO, 32>(mt) : block == 64 ? rows_entry<TI, TO, 64>(mt)
           : block == 128 ? rows_entry<TI, TO, 128>(mt) : nullptr;
}
template <class TI, class TO>
const QuantEntry *lookup_tile(int block) {
    static const QuantEntry e[3] = {{launch_tile<TI, TO, 32>, TM, TN, "quant_tile_128x128"},
                                    {launch_tile<TI, TO, 64>, TM, TN, "quant_tile_128x128"},
                                    {launch_tile<TI, TO, 128>, TM, TN, "quant_tile_128x128"}};
    return block == 32 ? &e[0] : block == 64 ? &e[1] : block == 128 ? &e[2] : nullptr;
}

}  // namespace

#if defined(TGE_PAIR_F16_F16)
const QuantEntry *quant_rows_f16_f16(int b, int mt) { return lookup_rows<TF16, OF16>(b, mt); }
const QuantEntry *quant_tile_f16_f16(int b) { return lookup_tile<TF16, OF16>(b); }
#elif defined(TGE_PAIR_F16_F32)
const QuantEntry *quant_rows_f16_f32(int b, int mt) { return lookup_rows<TF16, OF32>(b, mt); }
const QuantEntry *quant_tile_f16_f32(int b) { return lookup_tile<TF16, OF32>(b); }
#elif defined(TGE_PAIR_BF16_BF16)
const QuantEntry *quant_rows_bf16_bf16(int b, int mt) { return lookup_rows<TBF16, OBF16>(b, mt); }
const QuantEntry *quant_tile_bf16_bf16(int b) { return lookup_tile<TBF16, OBF16>(b); }
#elif defined(TGE_PAIR_BF16_F32)
const QuantEntry *quant_rows_bf16_f32(int b, int mt) { return lookup_rows<TBF16, OF32>(b, mt); }
const QuantEntry *quant_tile_bf16_f32(int b) { return lookup_tile<TBF16, OF32>(b); }
#else
#error "define one TGE_PAIR_* macro of a 16-bit float type"
#endif

}  // namespace tge
