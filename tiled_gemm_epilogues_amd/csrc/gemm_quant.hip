// Products with 4-bit weights on gfx950: D = act(alpha * A * W^T + beta * C + bias), where row n of
// W holds K codes q of 4 bits and, per block of G consecutive k, a scale s and a zero point z:
//
//   W[n][k] = s[n][k / G] * (q[n][k] - z[n][k / G])
//   D[m][n] = sum over blocks b of  s[n][b] * ( sum over k in b of  A[m][k] * (q[n][k] - z[n][b]) )
//
// The inner sums run on the matrix cores in the type of A, in which the small integers are exact,
// and the scale multiplies each block's sum in fp32: no weight is ever rounded.
//
// Codes become fp16 by bit operations: the 4 bits are set into the mantissa below the exponent of a
// power of two, which gives that power + q; one 32-bit word of 8 codes yields the pairs (k, k+4),
// k = 0 .. 3.  Then power + z is subtracted, so that the products are taken with q - z itself: -255
// .. 15, exact in fp16 and in bf16 (8 bits).  For fp16 that is one packed subtraction per pair.
// bf16 has no packed arithmetic: mixed-precision FMAs take the fp16 halves to fp32 differences, whose
// upper halves are packed, in the order of A's rows at no cost (17 instructions per word; fp16 12, and 4
// byte permutes for that order).  (bf16 sums of A * (16 + q) with (16 + z) * sum A subtracted take 7 per
// word and one more matrix instruction per A fragment, but cancel: weights that are all zero left
// rounding errors of sum A, and an infinite or very large A gave NaN.)
//
// A lane of a 16x16x32 matrix instruction holds 8 k of one weight row (n = lane % 16), its lane
// group g = lane / 16 saying which 8 of 32.  A 16-byte load of a lane covers 32 k of its row: lane
// group g holds k = 32g .. 32g+31 of a chunk of 128, while instruction i is to take k = 32i .. 32i+31
// (so that it stays inside one block, and a load of A's rows covers whole 64-byte pieces): word i
// of lane group g and word g of lane group i change places, a 4 x 4 transposition over the lane
// groups with two exchanges between the halves of the wave (permlane32_swap) and two between
// neighbouring groups (permlane16_swap).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"

namespace tge {
namespace {

using namespace dev;

constexpr int CHUNK = 128;    // k per step: 16 bytes of codes per lane

// the four words of a lane's 16 code bytes, transposed over the lane groups (see above)
__device__ __forceinline__ u32x4 exchange(u32x4 w) {
    const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{c[0], c[1], d[0], d[1]};
}

// 8 values of A in the order of the code pairs: (0,4) (1,5) (2,6) (3,7)
__device__ __forceinline__ u32x4 pair_order(u32x4 a) {
    return u32x4{__builtin_amdgcn_perm(a[2], a[0], 0x05040100u), __builtin_amdgcn_perm(a[2], a[0], 0x07060302u),
                 __builtin_amdgcn_perm(a[3], a[1], 0x05040100u), __builtin_amdgcn_perm(a[3], a[1], 0x07060302u)};
}

// Holds the mask in a scalar and the offset in a vector register, for one and-or instruction per
// pair (with literals it would be two).
__device__ __forceinline__ void in_registers(uint32_t &m, uint32_t &o) { asm("" : "+s"(m), "+v"(o)); }

typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// Per input type: what a block's zero point is held as (Off), and the values q - z of a word's codes,
// exact, as the pairs (0,4) (1,5) (2,6) (3,7) (PAIRS) or in the order of A's rows.
template <class TI>
struct Quant;
template <>
struct Quant<TF16> {
    using T = _Float16;
    static constexpr bool PAIRS = true;
    using Off = float;                                       // 16 + z
    __device__ static Off offset(float z) { return 16.0f + z; }
    __device__ static u32x4 values(uint32_t w, Off off) {
        uint32_t m = 0x03c003c0u, b = 0x4c004c00u;           // mantissa bits 6-9 of 16.0
        in_registers(m, b);
        u32x4 v = {((w << 6) & m) | b, ((w << 2) & m) | b, ((w >> 2) & m) | b, ((w >> 6) & m) | b};
        const _Float16 o = (_Float16)off;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = v[i];
            v[i] = __builtin_bit_cast(uint32_t, (h2)(__builtin_bit_cast(h2, x) - (h2){o, o}));
        }
        return v;
    }
};
template <>
struct Quant<TBF16> {
    using T = __bf16;
    static constexpr bool PAIRS = false;
    using Off = h2;                                          // -(1024 + z) and -(64 + z)
    __device__ static Off offset(float z) { return h2{(_Float16)(-1024.0f - z), (_Float16)(-64.0f - z)}; }
    // (the low halves are zero)
    __device__ static uint32_t pack(float a, float b) {
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
    }
    __device__ static u32x4 values(uint32_t w, Off off) {
        // codes at bits 0 and 16 are the lowest of the mantissas of 1024.0, those at bits 4 and 20 the
        // same of 64.0; codes 2, 3, 6 and 7 lie 8 bits further up
        uint32_t m0 = 0x000f000fu, b0 = 0x64006400u, m1 = 0x00f000f0u, b1 = 0x54005400u;
        in_registers(m0, b0);
        in_registers(m1, b1);
        float one = 1.0f;
        asm("" : "+v"(one));                                 // keeps the product: fma(half, one, half) is one instruction
        const uint32_t x[4] = {(w & m0) | b0, (w & m1) | b1, ((w >> 8) & m0) | b0, ((w >> 8) & m1) | b1};
        float lo[4], hi[4];                                  // codes i and i + 4
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const h2 h = __builtin_bit_cast(h2, x[i]);
            lo[i] = __builtin_fmaf((float)h[0], one, (float)off[i & 1]);
            hi[i] = __builtin_fmaf((float)h[1], one, (float)off[i & 1]);
        }
        return u32x4{pack(lo[0], lo[1]), pack(lo[2], lo[3]), pack(hi[0], hi[1]), pack(hi[2], hi[3])};
    }
};

// The values of a word in the order of A's rows: (0,1) (2,3) (4,5) (6,7)
template <class TI>
__device__ __forceinline__ u32x4 row_values(uint32_t w, typename Quant<TI>::Off off) {
    const u32x4 v = Quant<TI>::values(w, off);
    if constexpr (!Quant<TI>::PAIRS) return v;
    else return u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x05040100u),
                      __builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
}

// Scales and zero points of a weight row's blocks in one chunk.
template <class TI, int NBLK>
struct Blocks {
    float s[NBLK];
    typename Quant<TI>::Off off[NBLK];
};

// Eight consecutive scales (16 bytes) and zero points (8 bytes) of one weight row, as loaded; a
// scale load touches one cache line per row however few scales it takes, so eight at once.  Those
// past the row's end are zero.  Z: the weights have zero points (else every one is 8).
constexpr int SCALES = 8;
template <bool Z>
struct ScaleRegs {
    u32x4 s;
    uint2 z;
    __device__ __forceinline__ void load(const QuantParams &p, int64_t row, int b, int nblk) {
        const uint8_t *sp = static_cast<const uint8_t *>(p.scales) + (row + b) * 2;
        const uint8_t *zp = p.zeros + row + b;
        if (b + SCALES <= nblk) {
            s = ldg16(sp);
            if constexpr (Z) __builtin_memcpy(&z, zp, 8);
        } else {
            uint16_t v[SCALES];
            uint8_t w[SCALES];
#pragma unroll
            for (int i = 0; i < SCALES; ++i) {
                v[i] = 0;
                w[i] = 0;
                if (b + i < nblk) {
                    __builtin_memcpy(&v[i], sp + 2 * i, 2);
                    if constexpr (Z) w[i] = zp[i];
                }
            }
            __builtin_memcpy(&s, v, 16);
            if constexpr (Z) __builtin_memcpy(&z, w, 8);
        }
    }
};
// A row's eight in LDS (16 bytes of scales; 8 of zero points), and the NBLK from block i on.
template <class TI, int NBLK, bool Z>
__device__ __forceinline__ Blocks<TI, NBLK> read_blocks(const uint8_t *s, const uint8_t *z, int i) {
    using T = typename Quant<TI>::T;
    T v[NBLK];
    uint8_t w[NBLK];
    __builtin_memcpy(v, __builtin_assume_aligned(s + 2 * i, 2 * NBLK), sizeof v);
    if constexpr (Z) __builtin_memcpy(w, __builtin_assume_aligned(z + i, NBLK), sizeof w);
    Blocks<TI, NBLK> x;
#pragma unroll
    for (int b = 0; b < NBLK; ++b) {
        x.s[b] = (float)v[b];
        x.off[b] = Quant<TI>::offset(Z ? (float)w[b] : 8.0f);
    }
    return x;
}

// Adds one block's sum, times its scale, to the accumulator.
__device__ __forceinline__ void add_block(f32x4 &acc, f32x4 t, float s) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(s, t[e], acc[e]);
}

// 16 rows x 64 bytes in LDS: 16-byte piece q of row r.  Global loads take 4 consecutive lanes per
// row (lane / 4, lane % 4), so that the address unit sees whole 64-byte pieces (16 lanes on 16
// different rows cost four times as many cache accesses, which bound the first version of this
// kernel); a fragment takes row lane % 16, piece lane / 16.  LDS carries the data from one lane
// order to the other.  A 16-byte read serves lanes 0-3, 12-15, 20-23 and 24-27 together, then 4-11, 16-19
// and 28-31 (and 32 on likewise); with the pieces of row quads 0 .. 3 moved by swap16 = 0, 2, 3, 1
// their 16 places differ (bank conflicts of the tiles 4.8 M -> 0.65 M cycles, 102.3 -> 101.1 us;
// moved by 0, 1, 2, 3 half of the reads met).
__device__ __forceinline__ int swap16(int r) {
    const int t = r >> 2;
    return ((t << 1) & 2) ^ (t & 2 ? 3 : 0);
}
__device__ __forceinline__ int piece16(int r, int q) { return r * 64 + ((q ^ swap16(r)) << 4); }

// Orders this wave's LDS accesses (they execute in order; no instruction).
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The block that holds chunk ch (blocks of whole chunks): ch / (block / 128) by the reciprocal
// ceil(2^32 / (block / 128)), exact while the number of chunks is below 2^16.
__device__ __forceinline__ int block_of(const QuantParams &p, int ch) {
    return (int)((uint64_t)(uint32_t)ch * p.block_rcp >> 32);
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

// Eight columns of a row, nv of them inside N.
template <class T>
__device__ __forceinline__ void store_row(const QuantParams &p, int m, int n, int nv, const float (&sum)[8], const float (&bias)[8]) {
    const int64_t idx = (int64_t)m * p.ldc + n;
    const T *C = static_cast<const T *>(p.C) + idx;
    T *D = static_cast<T *>(p.D) + idx;
    T c[8], d[8];
    if (p.has_beta) {
        if (nv == 8) {
            __builtin_memcpy(c, C, sizeof c);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = C[min(e, nv - 1)];
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float x = p.alpha * sum[e];
        if (p.has_beta) x += p.beta * (float)c[e];
        x += bias[e];
        if (p.relu) x = x > 0.0f ? x : 0.0f;
        d[e] = (T)x;
    }
    if (nv == 8) {
        __builtin_memcpy(D, d, sizeof d);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < nv) D[e] = d[e];
    }
}

// Waits for this wave's loads, the direct ones (which the compiler does not count) too.
__device__ __forceinline__ void wait_all_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// ---- few rows ----------------------------------------------------------------------------------
// 16 rows and 16 * CG columns per workgroup, K divided over its WAVES waves; each wave reads its
// weights once, through registers (one chunk ahead) and a private LDS slot that only changes the
// lane order.  A comes from L2: every workgroup reads it, CG column groups share one reading.  The
// waves' sums are added through LDS in wave order.  Two workgroups fit a CU, so that one's loads
// are in flight while the other starts or ends.
//
// Bound by the weights' bytes, and below that by the latency of each wave's chunks, one ahead, and the
// conversion of the codes.  Measured, operands cold: 1 row, 4096 x 4096, block 128 (8.7 MB), bf16 6.3
// us, of which the launch 2.9; 16 rows, 16384 x 4096, block 64 with zero points, fp16 14.9 us (2.5 TB/s), bf16
// 15.5; 32 rows over 32 experts (20 of them used) of 2048 x 4096, block 128, bf16 29.5, fp16 27.3.  4 or 16
// waves and 32 columns measured no better, two chunks in flight slower (25.9 -> 32.5 for the last); 16
// columns take one row of 4096 x 4096 from 10.6 to 6.4 us (more workgroups), 64 columns 16 rows of 16384 x
// 4096 from 21.1 to 15.7 (A read less often).
constexpr int WAVES = 8;

template <class TI, class TO, int G, bool Z, int CG>
__global__ __launch_bounds__(WAVES * 64, 2) void quant_rows(QuantParams p) {
    using T = typename TO::T;
    using QT = Quant<TI>;
    constexpr int NBLK = G >= 128 ? 1 : CHUNK / G;           // blocks per chunk
    constexpr int SUB = 4 / NBLK;                            // matrix instructions per block
    constexpr int SC = SCALES / NBLK;                        // chunks per scale load
    constexpr int COLS = 16 * CG;
    // a wave's slot: codes, A, scales and zero points
    constexpr int OFF_A = CG * 1024, OFF_S = OFF_A + 4096, OFF_Z = OFF_S + COLS * 16;
    constexpr int SLOT = OFF_Z + (Z ? COLS * 8 : 0);
    static_assert(SLOT >= CG * 1024, "the slots hold the waves' sums at the end");
    __shared__ __attribute__((aligned(16))) uint8_t smem[WAVES * SLOT];
    struct Chunk {
        u32x4 q[CG], a[4];
    };

    int tn;
    if (!select_tile<(int)sizeof(T)>(p, 16, tn)) return;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane >> 2, lq = lane & 3;                 // load order: row, piece
    const int nch = (p.K + CHUNK - 1) / CHUNK, nblk = p.K / p.block;
    const int c0 = (int)((int64_t)nch * wave / WAVES), c1 = (int)((int64_t)nch * (wave + 1) / WAVES);
    const uint8_t *qrow[CG];
#pragma unroll
    for (int j = 0; j < CG; ++j) qrow[j] = p.Q + (int64_t)min(tn * COLS + 16 * j + lr, p.N - 1) * p.ldq;
    const uint8_t *arow = static_cast<const uint8_t *>(p.A) + (int64_t)min(lr, p.M - 1) * p.lda * 2;
    const int64_t srow = (int64_t)min(tn * COLS + lane, p.N - 1) * p.lds;
    uint8_t *const slot = smem + wave * SLOT;
    const int put = piece16(lr, lq), get = piece16(lane & 15, g);

    // The last chunk may end inside K (after whole blocks of 32): its loads stay in the row, and A
    // counts as zero past K.
    auto load = [&](Chunk &c, int ch) {
        const int k0 = ch * CHUNK;
        const int at = G >= 128 ? k0 / 2 + 16 * lq : min(k0 / 2 + 16 * lq, p.K / 2 - 16);
#pragma unroll
        for (int j = 0; j < CG; ++j) c.q[j] = ldg16(qrow[j] + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + 32 * i + 8 * lq;
            c.a[i] = ldg16(arow + 2 * (G >= 128 ? k : min(k, p.K - 8)));
        }
    };
    auto first_block = [&](int ch) { return G >= 128 ? block_of(p, ch) : ch * NBLK; };

    f32x4 acc[CG];
#pragma unroll
    for (int j = 0; j < CG; ++j) acc[j] = f32x4{0, 0, 0, 0};
    // chunk ch from registers to the slot, A in the order of the codes
    auto stage = [&](const Chunk &c, int ch) {
#pragma unroll
        for (int j = 0; j < CG; ++j) *reinterpret_cast<u32x4 *>(slot + 1024 * j + put) = c.q[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4 v = QT::PAIRS ? pair_order(c.a[i]) : c.a[i];
            if constexpr (G < 128) {   // an instruction's 32 k are inside K or past it
                if (ch * CHUNK + 32 * i >= p.K) v = u32x4{0, 0, 0, 0};
            }
            *reinterpret_cast<u32x4 *>(slot + OFF_A + 1024 * i + put) = v;
        }
    };
    // the chunk in the slot, its scales from index bi on
    auto compute = [&](int bi) {
        u32x4 w[CG];
        Blocks<TI, NBLK> blk[CG];
#pragma unroll
        for (int j = 0; j < CG; ++j) {
            const int row = 16 * j + (lane & 15);
            w[j] = exchange(*reinterpret_cast<const u32x4 *>(slot + 1024 * j + get));
            blk[j] = read_blocks<TI, NBLK, Z>(slot + OFF_S + 16 * row, slot + OFF_Z + 8 * row, bi);
        }
#pragma unroll
        for (int b = 0; b < NBLK; ++b) {
            f32x4 t[CG];
#pragma unroll
            for (int j = 0; j < CG; ++j) t[j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = b * SUB; i < (b + 1) * SUB; ++i) {
                const u32x4 a = *reinterpret_cast<const u32x4 *>(slot + OFF_A + 1024 * i + get);
#pragma unroll
                for (int j = 0; j < CG; ++j) t[j] = TI::mma16(a, QT::values(w[j][i], blk[j].off[b]), t[j]);
            }
#pragma unroll
            for (int j = 0; j < CG; ++j) add_block(acc[j], t[j], blk[j].s[b]);
        }
    };

    if (c0 < c1) {
        ScaleRegs<Z> sr;
        Chunk x;
        sr.load(p, srow, first_block(c0), nblk);
        load(x, c0);
        int base = 0, next = c0;                             // block at index 0 of the slot; chunk of new scales
#pragma unroll 1
        for (int ch = c0; ch < c1; ++ch) {
            wave_order();                                    // the last chunk's reads come first
            if (ch == next) {   // every SC chunks: scales loaded SC chunks ago to the slot
                base = first_block(ch);
                if (lane < COLS) {
                    *reinterpret_cast<u32x4 *>(slot + OFF_S + 16 * lane) = sr.s;
                    if constexpr (Z) *reinterpret_cast<uint2 *>(slot + OFF_Z + 8 * lane) = sr.z;
                }
                next += SC;
                if (next < c1) sr.load(p, srow, first_block(next), nblk);
            }
            stage(x, ch);
            wave_order();
            if (ch + 1 < c1) load(x, ch + 1);                // in flight while this chunk is computed
            compute(first_block(ch) - base);
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
    const int n = tn * COLS + 16 * wave + (lane & 15);
    if (n >= p.N) return;
    const float bias = p.has_bias ? static_cast<const float *>(p.bias)[n] : 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int m = 4 * g + r;
        if (m < p.M) store_one<T>(p, m, n, sum[r], bias);
    }
}

// ---- many rows ---------------------------------------------------------------------------------
// 128 x 128 output tile, 4 waves of 64 x 64, two workgroups per CU.  Chunks of 128 k of A go to LDS
// directly, the next one while this one is multiplied (two buffers, one barrier per chunk); each wave
// loads the codes of its own 64 columns in fragment order (4 loads, which share cache lines badly, but
// need no LDS) and brings its scales through a private slot.  A stays in its order, so the code
// pairs are brought into A's: permuting A instead would take it through registers, and all 256
// are in use.
//
// Bound by issue: of a chunk's instructions per wave (bf16, block 128) 64 are matrix ones (1024
// cycles) and some 350 vector ones (17 per word of codes, 1 per sum and block), shared by two
// waves per SIMD.  2048 x 4096 x 4096, operands cold, block 128 with zero points, bf16 101 us (0.68
// PFLOP/s), fp16 97, without them 95 and 92; block 32 130 and 129, 118 and 118.
// Earlier form, everything staged through registers and two barriers per chunk: 104 us.
constexpr int TM = 128, TN = 128, TNT = 256;

__device__ __forceinline__ uint32_t lds_addr(const uint8_t *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)p;
}

// direct-to-LDS 16-byte load per lane (LDS destination lds + 16 * lane), see gemm_fast.hip
__device__ __forceinline__ void dma16(const void *sbase, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %0"
                 :: "s"(sbase), "v"(voff), "s"(lds) : "memory", "m0");
}

template <class TI, class TO, int G, bool Z>
__global__ __launch_bounds__(TNT, 2) void quant_tile(QuantParams p) {
    using T = typename TO::T;
    using QT = Quant<TI>;
    constexpr int NBLK = G >= 128 ? 1 : CHUNK / G;
    constexpr int SUB = 4 / NBLK;
    constexpr int SC = SCALES / NBLK;
    // two buffers of A (8 groups of 16 rows x 4 pieces of 32 k); each wave's slot: codes of 32
    // columns, scales and zero points of 64 (replaced every SC chunks)
    constexpr int BUF = TM * CHUNK * 2, OFF_Z = 1024, SLOT = OFF_Z + (Z ? 512 : 0);
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * BUF + 4 * SLOT];

    int tn;
    if (!select_tile<(int)sizeof(T)>(p, TM, tn)) return;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int nch = (p.K + CHUNK - 1) / CHUNK, nblk = p.K / p.block;
    const int lr = lane >> 2, lq = lane & 3;
    const int put = piece16(lr, lq), get = piece16(lane & 15, g);
    uint8_t *const slot = smem + 2 * BUF + wave * SLOT;

    // A: this wave brings row groups 2w, 2w+1.  A direct load's lane writes position lane % 4 of row
    // lane / 4, where piece16 keeps piece lq ^ swap16(row).
    const uint8_t *const abase = dma_base<GROUP_ROWS>(p.A);
    const bool direct = ((reinterpret_cast<uintptr_t>(abase) | (uintptr_t)p.lda * 2) & 15) == 0 && p.lda < (1 << 23);
    int ar[2];
    uint32_t voff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        ar[i] = min(16 * (2 * wave + i) + lr, p.M - 1);
        voff[i] = (uint32_t)ar[i] * (uint32_t)p.lda * 2u + 16u * (uint32_t)(lq ^ swap16(lr));
    }
    auto bring = [&](int ch) {
        const int k0 = ch * CHUNK, buf = (ch & 1) * BUF + 8192 * wave;
        if (direct && k0 + CHUNK <= p.K) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    dma16(abase + 2 * (int64_t)(k0 + 32 * s), voff[i], lds_addr(smem) + buf + (4 * i + s) * 1024);
        } else {   // unaligned rows, or a chunk that ends inside K (after whole blocks): zeros past it
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int k = k0 + 32 * s;
                    u32x4 v = u32x4{0, 0, 0, 0};
                    if (k < p.K) v = ldg16(static_cast<const uint8_t *>(p.A) + ((int64_t)ar[i] * p.lda + k + 8 * lq) * 2);
                    *reinterpret_cast<u32x4 *>(smem + buf + (4 * i + s) * 1024 + put) = v;
                }
        }
    };
    // codes of this wave's 64 columns, 16 rows of 64 bytes each
    const uint8_t *qrow[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) qrow[j] = p.Q + (int64_t)min(tn * TN + wn * 64 + 16 * j + (lane & 15), p.N - 1) * p.ldq;
    u32x4 sq[4];
    auto fetch = [&](int ch) {
        const int at = ch * (CHUNK / 2) + 16 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) sq[j] = ldg16(qrow[j] + (G >= 128 ? at : min(at, p.K / 2 - 16)));
    };
    const int64_t srow = (int64_t)min(tn * TN + wn * 64 + lane, p.N - 1) * p.lds;
    auto first_block = [&](int ch) { return G >= 128 ? block_of(p, ch) : ch * NBLK; };

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    int base = 0, next = 0;                                  // block at index 0 of the scales; chunk of new ones
    if (nch > 0) {
        fetch(0);
        bring(0);
    }
#pragma unroll 1
    for (int ch = 0; ch < nch; ++ch) {
        wait_all_loads();                                    // this chunk's A, for every wave after the barrier
        u32x4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = exchange(sq[j]);
        __syncthreads();                                     // (and the other buffer's reads are done)
        if (ch + 1 < nch) bring(ch + 1);
        if (ch == next) {
            base = first_block(ch);
            // loaded here and not ahead: the registers to hold them are not there (spilled 105 us, 99 so)
            ScaleRegs<Z> sr;
            sr.load(p, srow, base, nblk);
            wave_order();
            *reinterpret_cast<u32x4 *>(slot + 16 * lane) = sr.s;
            if constexpr (Z) *reinterpret_cast<uint2 *>(slot + OFF_Z + 8 * lane) = sr.z;
            next += SC;
        }
        const int bi = first_block(ch) - base;
        Blocks<TI, NBLK> blk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 16 * j + (lane & 15);
            blk[j] = read_blocks<TI, NBLK, Z>(slot + 16 * row, slot + OFF_Z + 8 * row, bi);
        }
        const uint8_t *const la = smem + (ch & 1) * BUF + wm * 16384 + get;
        // Steps of 4 matrix instructions (one word of codes against 4 row groups).  Beside them run the
        // conversion of the next step's word and the scaling of the column group before.
        u32x4 v = row_values<TI>(w[0][0], blk[0].off[0]);
        f32x4 tp[4];
#pragma unroll
        for (int b = 0; b < NBLK; ++b) {
            u32x4 a[4][SUB];
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i][s] = *reinterpret_cast<const u32x4 *>(la + (4 * i + b * SUB + s) * 1024);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 t[4];
                if (b == NBLK - 1 && j == 2) fetch(min(ch + 1, nch - 1));   // (no branch: the last again)
#pragma unroll
                for (int s = 0; s < SUB; ++s) {
                    // next word: (s + 1, j), (0, j + 1) or the next block's first
                    const int nj = s + 1 < SUB ? j : (j + 1) & 3, ns = s + 1 < SUB ? s + 1 : 0;
                    const int nb = s + 1 < SUB || j < 3 ? b : b + 1;
                    u32x4 nv = v;
                    if (nb < NBLK) nv = row_values<TI>(w[nj][nb * SUB + ns], blk[nj].off[nb]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[i] = TI::mma16(a[i][s], v, s ? t[i] : f32x4{0, 0, 0, 0});
                    if (j > 0 || b > 0) {
                        const int pj = (j + 3) & 3, pb = j > 0 ? b : b - 1;
#pragma unroll
                        for (int i = s * 4 / SUB; i < (s + 1) * 4 / SUB; ++i)
                            add_block(acc[i][pj], tp[i], blk[pj].s[pb]);
                    }
                    v = nv;
                    // one matrix instruction, then the vector ones that fit beside it
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x2, SUB == 4 ? 5 : SUB == 2 ? 7 : 11, 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) tp[i] = t[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) add_block(acc[i][3], tp[i], blk[3].s[NBLK - 1]);
    }

    // The sums go through LDS, so that a store covers whole rows of 64 columns (8 lanes of 8 columns);
    // 2-byte stores by the accumulators' layout took 3 us more (2048 x 4096 x 4096).
    __syncthreads();
    constexpr int STR = 68;                                  // floats between rows: no bank is met twice
    float *const st = reinterpret_cast<float *>(smem) + wave * 16 * STR;
    const int er = lane >> 3, ec = 8 * (lane & 7), n = tn * TN + wn * 64 + ec;
    const int nv = min(p.N - n, 8);                          // columns of this lane
    float bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = p.has_bias && nv > 0 ? static_cast<const float *>(p.bias)[n + min(e, nv - 1)] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        wave_order();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) st[(4 * g + r) * STR + 16 * j + (lane & 15)] = acc[i][j][r];
        wave_order();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[8];
            __builtin_memcpy(x, __builtin_assume_aligned(st + (8 * h + er) * STR + ec, 16), sizeof x);
            const int m = wm * 64 + 16 * i + 8 * h + er;
            if (m < p.M && nv > 0) store_row<T>(p, m, n, nv, x, bias);
        }
    }
}

// ---- entries -----------------------------------------------------------------------------------

template <class TI, class TO, int G, int CG>
hipError_t launch_rows(const QuantParams &p, unsigned grid, hipStream_t s) {
    if (p.zeros) hipLaunchKernelGGL((quant_rows<TI, TO, G, true, CG>), dim3(grid), dim3(WAVES * 64), 0, s, p);
    else hipLaunchKernelGGL((quant_rows<TI, TO, G, false, CG>), dim3(grid), dim3(WAVES * 64), 0, s, p);
    return hipGetLastError();
}
template <class TI, class TO, int G>
hipError_t launch_tile(const QuantParams &p, unsigned grid, hipStream_t s) {
    if (p.zeros) hipLaunchKernelGGL((quant_tile<TI, TO, G, true>), dim3(grid), dim3(TNT), 0, s, p);
    else hipLaunchKernelGGL((quant_tile<TI, TO, G, false>), dim3(grid), dim3(TNT), 0, s, p);
    return hipGetLastError();
}

template <class TI, class TO>
const QuantEntry *lookup_rows(int block, int cg) {
    static const QuantEntry e[6] = {{launch_rows<TI, TO, 32, 1>, 16, 16, "quant_rows_16x16"},
                                    {launch_rows<TI, TO, 32, 4>, 16, 64, "quant_rows_16x64"},
                                    {launch_rows<TI, TO, 64, 1>, 16, 16, "quant_rows_16x16"},
                                    {launch_rows<TI, TO, 64, 4>, 16, 64, "quant_rows_16x64"},
                                    {launch_rows<TI, TO, 128, 1>, 16, 16, "quant_rows_16x16"},
                                    {launch_rows<TI, TO, 128, 4>, 16, 64, "quant_rows_16x64"}};
    if ((cg != 1 && cg != 4) || (block != 32 && block != 64 && block != 128)) return nullptr;
    return &e[(block == 32 ? 0 : block == 64 ? 2 : 4) + (cg == 4)];
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
const QuantEntry *quant_rows_f16_f16(int b, int cg) { return lookup_rows<TF16, OF16>(b, cg); }
const QuantEntry *quant_tile_f16_f16(int b) { return lookup_tile<TF16, OF16>(b); }
#elif defined(TGE_PAIR_F16_F32)
const QuantEntry *quant_rows_f16_f32(int b, int cg) { return lookup_rows<TF16, OF32>(b, cg); }
const QuantEntry *quant_tile_f16_f32(int b) { return lookup_tile<TF16, OF32>(b); }
#elif defined(TGE_PAIR_BF16_BF16)
const QuantEntry *quant_rows_bf16_bf16(int b, int cg) { return lookup_rows<TBF16, OBF16>(b, cg); }
const QuantEntry *quant_tile_bf16_bf16(int b) { return lookup_tile<TBF16, OBF16>(b); }
#elif defined(TGE_PAIR_BF16_F32)
const QuantEntry *quant_rows_bf16_f32(int b, int cg) { return lookup_rows<TBF16, OF32>(b, cg); }
const QuantEntry *quant_tile_bf16_f32(int b) { return lookup_tile<TBF16, OF32>(b); }
#else
#error "define one TGE_PAIR_* macro of a 16-bit float type"
#endif

}  // namespace tge
