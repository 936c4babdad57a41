// Layer norm over rows of up to 64 KiB and its gradients, for gfx950.
//
//   y = (x - m) r w + b,   m = mean of the row, r = 1 / sqrt(mean of (x - m)^2 + eps)
//   with h = (x - m) r and g = dy w:  dx = r (g - mean(g) - h mean(g h)) + beta C,
//   dw = sum over rows of dy h,  db = sum over rows of dy
//
// Bound by bytes: x in and y out, or dy, x (and C) in and dx out.  So a row stays in its team's
// registers between the sums and the result, each byte moves once, and the next row of a team is on
// its way while this one is worked on.  Short rows share a wave: 46547 rows of 64 fp16 16.5 -> 4.5 us, their
// gradient 26.6 -> 9.8.  Weight, bias and, in the gradient, the column sums stay in
// registers over all rows of a team.
//
// Statistics in fp32: a wave takes the mean and the squared deviations from it over its own part
// (two passes over registers, so nothing cancels), and the parts are joined by their means:
// M2 = sum of M2_w + n_w (m_w - m)^2.  So a row needs one exchange between its waves.
//
// Column sums: each team adds its rows up in registers, the teams of a workgroup are joined through
// LDS, and each workgroup writes one partial sum per column; norm_join adds them up.  All orders are
// fixed (no atomics): equal inputs give equal bits.
//
// Measured: 16384 rows of 8192 bf16 97 us (5.5 TB/s), the gradient of 16384 rows of 4096 with C and both sums
// 105 us (5.1 TB/s), of 5003 rows of 1001 fp16 14.6 us (two launches, 5 rows to a team); 7 rows of 4096 3.4 us.
// Rows of more than 32 KiB fill the registers of 16 waves: 300 of 24576 bf16 10.5 us, their gradient 80 (it spills).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"

namespace tge {
namespace {

using namespace dev;

// A lane's part of a row: C chunks of VE elements.  Chunk c stands at column n = (c W 64 + lane) VE; one
// that would cross the row's end is moved back to end with it, and its first `skip` elements, which the lane
// before has too, count for nothing: they are left out of sums, and stored twice with equal values.
// So no load or store is narrower than 16 bytes, unless the row is (SHORT: it may be).
template <class T, int W, int C>
struct Part {
    static constexpr int ES = (int)sizeof(T), VE = 16 / ES;
    static constexpr bool SHORT = W * C == 1;
    uint32_t col[C];         // (unsigned: a scalar row pointer and a 32-bit offset make an address)
    int skip[C];             // >= VE: outside the row
    bool whole[C];           // (uniform) no chunk of the wave is moved
    int n;                   // SHORT: the row's elements where they are fewer than a chunk's, else VE

    __device__ __forceinline__ static int column(int lane, int c) { return (c * W * 64 + lane) * VE; }
    // lane: of the row's (L of them in a wave)
    template <int L>
    __device__ __forceinline__ void init(int lane, int wave, int N) {
        n = SHORT ? min(N, VE) : VE;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = column(lane, c);
            const int from = max(min(at, N - VE), 0);
            col[c] = (uint32_t)from;
            skip[c] = at - from;
            whole[c] = column(wave * 64 + L, c) <= N;
            if (SHORT && n < VE) skip[c] = lane == 0 ? 0 : VE;
        }
    }
    __device__ __forceinline__ bool counts(int c, int e) const { return e >= skip[c] && (!SHORT || e < n); }
    __device__ __forceinline__ u32x4 load(const T *row, int c) const {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(row) + col[c] * (uint32_t)ES;
        if constexpr (SHORT) {
            if (n < VE) return ldg16_partial<ES>(p, skip[c] ? 0 : n);
        }
        return ldg16(p);
    }
    __device__ __forceinline__ void store(T *row, int c, const float *v) const {
        T out[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) out[e] = (T)v[e];
        if (skip[c] >= VE) return;
        if (SHORT && n < VE) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (e < n) row[col[c] + e] = out[e];
        } else {
            __builtin_memcpy(reinterpret_cast<uint8_t *>(row) + col[c] * (uint32_t)ES, out, 16);
        }
    }
    // its columns' sums (those of a moved chunk that another lane has too are the same there)
    __device__ __forceinline__ void store_sums(float *to, int c, const float (&v)[VE]) const {
        if (skip[c] >= VE) return;
        if (SHORT && n < VE) {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (e < n) to[col[c] + e] = v[e];
        } else {
            __builtin_memcpy(reinterpret_cast<uint8_t *>(to) + col[c] * 4u, v, sizeof(v));
        }
    }
    // its columns of weight or bias (`none` each without them)
    __device__ __forceinline__ void columns(float (&to)[VE], const float *v, int c, float none) const {
        if (!v) {
#pragma unroll
            for (int e = 0; e < VE; ++e) to[e] = none;
        } else if (SHORT && n < VE) {
#pragma unroll
            for (int e = 0; e < VE; ++e) to[e] = v[min(e, n - 1)];
        } else {
            __builtin_memcpy(to, reinterpret_cast<const uint8_t *>(v) + col[c] * 4u, sizeof(to));
        }
    }
};

// v, which the compiler does not see to be the same in every turn of a loop: what is loaded from there is
// loaded again, rather than held in registers throughout.
__device__ __forceinline__ int renewed(int v) {
    asm volatile("" : "+s"(v));
    return v;
}

// The chunk's words stand as they are from here on: values taken from them before are taken again
// rather than kept (16 registers of fp32 for 8 of pairs).
__device__ __forceinline__ void forget(u32x4 &v) { asm volatile("" : "+v"(v)); }
// One chunk's values at a time: work on several of them at once needs more registers than there are.
__device__ __forceinline__ void chunk_done() { __builtin_amdgcn_sched_barrier(0); }

template <class T>
__device__ __forceinline__ float element(const u32x4 &v, int e) {
    T t[16 / sizeof(T)];
    __builtin_memcpy(t, &v, 16);
    return (float)t[e];
}
// L: lanes of a row in a wave; with fewer than 64, a wave (of one) has 64 / L rows at a time.
template <class T, int W, int C, int TEAMS, int L>
__global__ __launch_bounds__(W * 64 * TEAMS) void norm_forward(NormParams p) {
    using P = Part<T, W, C>;
    constexpr int VE = P::VE;
    // the longest rows fill the registers: weight and bias come from the caches, rows when needed
    constexpr bool KEEP = C <= 2;
    __shared__ float slots[2][TEAMS][W][2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wave / W, tw = wave % W;
    const int lane = threadIdx.x - team * W * 64;
    static_assert(L == 64 || (W == 1 && C == 1), "several rows to a wave: of one chunk per lane");
    constexpr int R = 64 / L;
    const int l = L == 64 ? lane : lane % L, beside = L == 64 ? 0 : lane / L;
    const int N = p.N;
    const T *X = static_cast<const T *>(p.X);
    T *Y = static_cast<T *>(p.Y);
    P part;
    part.template init<L>(l, tw, N);

    // elements of this wave's part of a row
    int mine = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) mine += min(max(N - P::column(tw * 64, c), 0), 64 * VE);
    const float rn_w = mine ? 1.0f / (float)mine : 0.0f;
    // and of wave `wl`
    const int wl = threadIdx.x & 63;
    float nv = 0.0f;
    if constexpr (W > 1) {
        int n = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) n += min(max(N - P::column(wl * 64, c), 0), 64 * VE);
        nv = wl < W ? (float)n : 0.0f;
    }
    float w[KEEP ? C : 1][VE], b[KEEP ? C : 1][VE];
    if constexpr (KEEP) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            part.columns(w[c], p.weight, c, 1.0f);
            part.columns(b[c], p.bias, c, 0.0f);
        }
    }

    const int step = gridDim.x * TEAMS * R;
    int row = (blockIdx.x * TEAMS + team) * R + beside;
    u32x4 next[C];
    auto fetch = [&](int r) {
#pragma unroll
        for (int c = 0; c < C; ++c) next[c] = part.load(X + (int64_t)r * p.ldx, c);
    };
    if (KEEP && row < p.rows) fetch(row);
    int flip = 0;
    // the workgroup's first team has a row in every pass, so that all meet at the barriers
#pragma unroll 1
    for (int first = blockIdx.x * TEAMS * R; first < p.rows; first += step, row += step, flip ^= 1) {
        if (!KEEP && row < p.rows) fetch(row);
        u32x4 x[C];
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = next[c];
        if (KEEP && p.rows - row > step) fetch(row + step);
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (part.whole[c]) {
#pragma unroll
                for (int e = 0; e < VE; ++e) s += element<T>(x[c], e);
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) s += part.counts(c, e) ? element<T>(x[c], e) : 0.0f;
            }
        }
        float m = side_sum<L>(s) * rn_w, q = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (part.whole[c]) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float d = element<T>(x[c], e) - m;
                    q = __builtin_fmaf(d, d, q);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float d = part.counts(c, e) ? element<T>(x[c], e) - m : 0.0f;
                    q = __builtin_fmaf(d, d, q);
                }
            }
        }
        q = side_sum<L>(q);
        if constexpr (W > 1) {
            if ((lane & 63) == 0) {
                slots[flip][team][tw][0] = m;
                slots[flip][team][tw][1] = q;
            }
            __syncthreads();
            // lane v has wave v's
            const float mv = wl < W ? slots[flip][team][wl < W ? wl : 0][0] : 0.0f;
            const float qv = wl < W ? slots[flip][team][wl < W ? wl : 0][1] : 0.0f;
            const float mean = wave_sum(mv * (nv * p.rn)), d = mv - mean;
            q = wave_sum(__builtin_fmaf(nv * d, d, qv));
            m = mean;
        }
        const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(q, p.rn, p.eps));
        if (row < p.rows) {
#pragma unroll
            for (int c = 0; c < C; ++c) forget(x[c]);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                constexpr bool K = KEEP;
                float (&wc)[VE] = w[K ? c : 0], (&bc)[VE] = b[K ? c : 0];
                if (!K) {
                    part.columns(wc, p.weight + renewed(0), c, 1.0f);
                    part.columns(bc, p.bias + renewed(0), c, 0.0f);
                }
                float y[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) y[e] = __builtin_fmaf((element<T>(x[c], e) - m) * r, wc[e], bc[e]);
                part.store(Y + (int64_t)row * p.ldy, c, y);
            }
            if (l == 0) {
                if (p.mean) p.mean[row] = m;
                if (p.rstd) p.rstd[row] = r;
            }
        }
    }
}

template <class T, int W, int C, int TEAMS, int L>
__global__ __launch_bounds__(W * 64 * TEAMS) void norm_grad(NormParams p) {
    using P = Part<T, W, C>;
    constexpr int VE = P::VE;
    // as in the forward pass; 16 waves leave 128 registers each, too few for two kept chunks of 8 (300 rows of 16384
    // bf16, dX alone: 9.2 us so, 22.6 with them spilled)
    constexpr bool KEEP = C <= 2 && (W < 16 || VE < 8);
    __shared__ float slots[2][TEAMS][W][2];
    // the column sums of the teams, one half (weight, bias) after the other
    __shared__ float sums[TEAMS > 1 ? (TEAMS - 1) * W * 64 * VE * C : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wave / W, tw = wave % W;
    const int lane = threadIdx.x - team * W * 64;
    static_assert(L == 64 || (W == 1 && C == 1), "several rows to a wave: of one chunk per lane");
    constexpr int R = 64 / L;
    const int l = L == 64 ? lane : lane % L, beside = L == 64 ? 0 : lane / L;
    const int N = p.N;
    const T *X = static_cast<const T *>(p.X), *dY = static_cast<const T *>(p.Y), *Cm = static_cast<const T *>(p.C);
    T *dX = static_cast<T *>(p.dX);
    P part;
    part.template init<L>(l, tw, N);
    float w[KEEP ? C : 1][VE];
    if constexpr (KEEP) {
#pragma unroll
        for (int c = 0; c < C; ++c) part.columns(w[c], p.weight, c, 1.0f);
    }
    float dw[C][VE], db[C][VE];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < VE; ++e) dw[c][e] = db[c][e] = 0.0f;

    const int step = gridDim.x * TEAMS * R;
    int row = (blockIdx.x * TEAMS + team) * R + beside;
    u32x4 nx[C], ny[C];
    float nm = 0.0f, nr = 0.0f;
    auto clear = [&]() {
#pragma unroll
        for (int c = 0; c < C; ++c) nx[c] = ny[c] = u32x4{0, 0, 0, 0};
        nm = nr = 0.0f;
    };
    auto fetch = [&](int r) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            nx[c] = part.load(X + (int64_t)r * p.ldx, c);
            ny[c] = part.load(dY + (int64_t)r * p.ldy, c);
        }
        nm = p.mean[r];
        nr = p.rstd[r];
    };
    clear();
    if (KEEP && row < p.rows) fetch(row);
    int flip = 0;
#pragma unroll 1
    for (int first = blockIdx.x * TEAMS * R; first < p.rows; first += step, row += step, flip ^= 1) {
        const bool on = row < p.rows;
        if (!KEEP) fetch(row);               // (one team: it has a row)
        u32x4 x[C], y[C], res[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            x[c] = nx[c];
            y[c] = ny[c];
        }
        const float m = nm, r = nr;
        if (KEEP && p.has_beta && on) {
#pragma unroll
            for (int c = 0; c < C; ++c) res[c] = part.load(Cm + (int64_t)row * p.ldx, c);
        }
        // a team past the last row sums nothing
        if (KEEP) {
            if (p.rows - row > step) fetch(row + step);
            else clear();
        }
        float sg = 0.0f, sgh = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float (&wc)[VE] = w[KEEP ? c : 0];
            if (!KEEP) part.columns(wc, p.weight + renewed(0), c, 1.0f);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float dy = element<T>(y[c], e), h = (element<T>(x[c], e) - m) * r;
                // (elements that do not count add to column sums that are not stored)
                const float g = part.whole[c] || part.counts(c, e) ? dy * wc[e] : 0.0f;
                sg += g;
                sgh = __builtin_fmaf(g, h, sgh);
                dw[c][e] = __builtin_fmaf(dy, h, dw[c][e]);
                db[c][e] += dy;
            }
            chunk_done();
        }
        sg = side_sum<L>(sg);
        sgh = side_sum<L>(sgh);
        if constexpr (W > 1) {
            if ((lane & 63) == 0) {
                slots[flip][team][tw][0] = sg;
                slots[flip][team][tw][1] = sgh;
            }
            __syncthreads();
            // lane v has wave v's (all of them in every lane take 2 W registers at the worst place)
            const int wl = threadIdx.x & 63;
            sg = wave_sum(wl < W ? slots[flip][team][wl < W ? wl : 0][0] : 0.0f);
            sgh = wave_sum(wl < W ? slots[flip][team][wl < W ? wl : 0][1] : 0.0f);
        }
        sg *= p.rn;
        sgh *= p.rn;
        if (on) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                forget(x[c]);
                forget(y[c]);
                if (!KEEP && p.has_beta) res[c] = part.load(Cm + (int64_t)row * p.ldx, c);
            }
            // C may be dX: the chunk that is moved back shares columns with the lane before, which may be in
            // another wave (the other loads stand before the row's exchange)
            if (!KEEP && p.has_beta) __syncthreads();
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float (&wc)[VE] = w[KEEP ? c : 0];
                if (!KEEP) part.columns(wc, p.weight + renewed(0), c, 1.0f);
                float d[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float dy = element<T>(y[c], e), h = (element<T>(x[c], e) - m) * r;
                    d[e] = r * (__builtin_fmaf(dy, wc[e], -sg) - h * sgh);
                    if (p.has_beta) d[e] = __builtin_fmaf(p.beta, element<T>(res[c], e), d[e]);
                }
                part.store(dX + (int64_t)row * p.ldx, c, d);
                chunk_done();
            }
        }
    }
    if (!p.part) return;
    // one partial sum per column and workgroup: the rows side by side in a wave, then the teams
#pragma unroll
    for (int h = L; h < 64; h *= 2)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            dw[0][e] += __shfl_xor(dw[0][e], h);
            db[0][e] += __shfl_xor(db[0][e], h);
        }
    float *out = p.part + (int64_t)blockIdx.x * 2 * N;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if constexpr (TEAMS > 1) {
            constexpr int LANES = W * 64;
            __syncthreads();
            if (team > 0) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        sums[((team - 1) * C * VE + c * VE + e) * LANES + lane] = half ? db[c][e] : dw[c][e];
            }
            __syncthreads();
            if (team == 0) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        float t = half ? db[c][e] : dw[c][e];
#pragma unroll
                        for (int k = 1; k < TEAMS; ++k) t += sums[((k - 1) * C * VE + c * VE + e) * LANES + lane];
                        (half ? db[c][e] : dw[c][e]) = t;
                    }
            }
        }
        if (team == 0 && beside == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) part.store_sums(out + half * N, c, half ? db[c] : dw[c]);
        }
    }
}

#if defined(TGE_TYPE_F32)
// Sum over the workgroups' partial sums: NORM_SUM_COLS columns of 2 N per workgroup, 8 partial sums
// at a time, joined through LDS.
__global__ __launch_bounds__(256) void join(const float *part, int count, int N, float *dweight, float *dbias) {
    __shared__ float sums[256];
    const int c = threadIdx.x % NORM_SUM_COLS, r = threadIdx.x / NORM_SUM_COLS;
    constexpr int R = 256 / NORM_SUM_COLS;
    const int64_t n = (int64_t)blockIdx.x * NORM_SUM_COLS + c;
    float s = 0.0f;
    if (n < 2 * (int64_t)N) {
#pragma unroll 8
        for (int i = r; i < count; i += R) s += part[(int64_t)i * 2 * N + n];
    }
    sums[threadIdx.x] = s;
    __syncthreads();
    if (r > 0 || n >= 2 * (int64_t)N) return;
#pragma unroll
    for (int k = 1; k < R; ++k) s += sums[k * NORM_SUM_COLS + c];
    if (n < N) {
        if (dweight) dweight[n] = s;
    } else if (dbias) {
        dbias[n - N] = s;
    }
}
#endif

template <class T, int W, int C, int TEAMS, int L, bool GRAD>
hipError_t launch(const NormParams &p, unsigned grid, hipStream_t stream) {
    if constexpr (GRAD) hipLaunchKernelGGL((norm_grad<T, W, C, TEAMS, L>), dim3(grid), dim3(W * 64 * TEAMS), 0, stream, p);
    else hipLaunchKernelGGL((norm_forward<T, W, C, TEAMS, L>), dim3(grid), dim3(W * 64 * TEAMS), 0, stream, p);
    return hipGetLastError();
}

template <class T, bool GRAD>
hipError_t by_shape(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream) {
#define TGE_NORM_CASE(W, C, L) \
    case ((W) * 8 + (C)) * 64 + (L) - 1: return launch<T, W, C, norm_teams(W, GRAD), L, GRAD>(p, grid, stream)
    if (s.teams != norm_teams(s.waves, GRAD)) return hipErrorInvalidValue;
    switch ((s.waves * 8 + s.chunks) * 64 + s.lanes - 1) {
        TGE_NORM_CASE(1, 1, 8);
        TGE_NORM_CASE(1, 1, 16);
        TGE_NORM_CASE(1, 1, 32);
        TGE_NORM_CASE(1, 1, 64);
        TGE_NORM_CASE(1, 2, 64);
        TGE_NORM_CASE(2, 2, 64);
        TGE_NORM_CASE(3, 2, 64);
        TGE_NORM_CASE(4, 2, 64);
        TGE_NORM_CASE(6, 2, 64);
        TGE_NORM_CASE(8, 2, 64);
        TGE_NORM_CASE(12, 2, 64);
        TGE_NORM_CASE(16, 2, 64);
        TGE_NORM_CASE(16, 3, 64);
        TGE_NORM_CASE(16, 4, 64);
    default: return hipErrorInvalidValue;
    }
#undef TGE_NORM_CASE
}

}  // namespace

#if defined(TGE_TYPE_F32)
hipError_t norm_forward_f32(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return by_shape<float, false>(p, s, g, st); }
hipError_t norm_grad_f32(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return by_shape<float, true>(p, s, g, st); }

hipError_t norm_join(const float *part, int count, int N, float *dweight, float *dbias, hipStream_t stream) {
    const unsigned grid = (unsigned)((2 * (int64_t)N + NORM_SUM_COLS - 1) / NORM_SUM_COLS);
    hipLaunchKernelGGL(join, dim3(grid), dim3(256), 0, stream, part, count, N, dweight, dbias);
    return hipGetLastError();
}
#elif defined(TGE_TYPE_F16)
hipError_t norm_forward_f16(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return by_shape<_Float16, false>(p, s, g, st); }
hipError_t norm_grad_f16(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return by_shape<_Float16, true>(p, s, g, st); }
#elif defined(TGE_TYPE_BF16)
hipError_t norm_forward_bf16(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return by_shape<__bf16, false>(p, s, g, st); }
hipError_t norm_grad_bf16(const NormParams &p, NormShape s, unsigned g, hipStream_t st) { return by_shape<__bf16, true>(p, s, g, st); }
#else
#error "define one TGE_TYPE_* macro"
#endif

}  // namespace tge
