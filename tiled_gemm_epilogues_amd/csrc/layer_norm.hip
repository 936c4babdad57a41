// Layer norm over rows of up to 64 KiB and its gradients, for gfx950.
//
//   y = (x - m) r w + b,   m = mean of the row, r = 1 / sqrt(mean of (x - m)^2 + eps)
//   with h = (x - m) r and g = dy w:  dx = r (g - mean(g) - h mean(g h)) + beta C,
//   dw = sum over rows of dy h,  db = sum over rows of dy
//
// Bound by bytes: x in and y out, or dy, x (and C) in and dx out.  So a row stays in its team's
// registers between the sums and the result, each byte moves once, and the next row of a team is on
// its way while this one is worked on.  Weight, bias and, in the gradient, the column sums stay in
// registers over all rows of a team.
//
// Statistics in fp32: a wave takes the mean and the squared deviations from it over its own part
// (two passes over registers, so nothing cancels), and the parts are joined by their means:
// M2 = sum of M2_w + n_w (m_w - m)^2.  So a row needs one exchange between its waves.
//
// Column sums: each team adds its rows up in registers, the teams of a workgroup are joined through
// LDS, and each workgroup writes one partial sum per column; norm_join adds them up.  All orders are
// fixed (no atomics): equal inputs give equal bits.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"

namespace tge {
namespace {

using namespace dev;

// Sum over the wave's 64 lanes, in every lane (scalar): the data-parallel lane moves of
// wave_scan_add.
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

// A lane's part of a row: C chunks of VE elements from columns col(c) on.
template <class T, int W, int C>
struct Part {
    static constexpr int VE = 16 / (int)sizeof(T);
    __device__ __forceinline__ static int col(int lane, int c) { return (c * W * 64 + lane) * VE; }
};

// Chunk at column n of a row, zero past its N elements.  whole: every chunk of the wave lies inside
// the row.  Else a load that ends with the row at the latest, moved down, so that no lane branches;
// SHORT: the row may be shorter than a chunk.
template <class T, bool SHORT>
__device__ __forceinline__ u32x4 load_chunk(const T *row, int n, int N, bool whole) {
    constexpr int ES = (int)sizeof(T), VE = 16 / ES;
    if (whole) return ldg16(reinterpret_cast<const uint8_t *>(row + n));
    if constexpr (SHORT) {
        if (N < VE) return ldg16_partial<ES>(reinterpret_cast<const uint8_t *>(row + min(n, N)), N - n);
    }
    const int at = min(n, N - VE), past = n - at;
    const u32x4 v = ldg16(reinterpret_cast<const uint8_t *>(row + at));
    uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    if (past * ES >= 8) {
        lo = hi;
        hi = 0;
    }
    const int bits = 8 * (past * ES & 7);
    lo = lo >> bits | (bits ? hi << (64 - bits) : 0);
    hi >>= bits;
    if (past >= VE) lo = 0;
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
template <class T>
__device__ __forceinline__ void store_chunk(T *row, int n, int N, bool whole, const float *v) {
    constexpr int ES = (int)sizeof(T), VE = 16 / ES;
    T out[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) out[e] = (T)v[e];
    if (whole || n + VE <= N) {
        __builtin_memcpy(row + n, out, 16);
    } else if (n < N) {                  // the row's last elements, in pieces of 4, 2 and 1
        const int have = N - n;
        uint8_t *to = reinterpret_cast<uint8_t *>(row + n);
        uint64_t w[2];
        __builtin_memcpy(w, out, 16);
        if (have * ES & 8) {
            __builtin_memcpy(to, &w[0], 8);
            w[0] = w[1];
            to += 8;
        }
        if (have * ES & 4) {
            const uint32_t x = (uint32_t)w[0];
            __builtin_memcpy(to, &x, 4);
            w[0] >>= 32;
            to += 4;
        }
        if (have * ES & 2) {
            const uint16_t x = (uint16_t)w[0];
            __builtin_memcpy(to, &x, 2);
        }
    }
}
// A value of the row's loop that the compiler does not see to be the same in every turn: what is
// derived from it is derived again, rather than held in registers (masks of every element) throughout.
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
// VE columns of weight or bias from n on (`none` each without them); past N the last one's, for
// values that are not used.
template <int VE>
__device__ __forceinline__ void load_columns(float (&to)[VE], const float *v, int n, int N, bool whole, float none) {
    if (!v) {
#pragma unroll
        for (int e = 0; e < VE; ++e) to[e] = none;
    } else if (whole) {
        __builtin_memcpy(to, v + n, sizeof(to));
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) to[e] = v[min(n + e, N - 1)];
    }
}

template <class T, int W, int C, int TEAMS>
__global__ __launch_bounds__(W * 64 * TEAMS) void norm_forward(NormParams p) {
    using P = Part<T, W, C>;
    constexpr int VE = P::VE;
    // the longest rows fill the registers: weight and bias come from the caches, rows when needed
    constexpr bool KEEP = C <= 2;
    __shared__ float slots[2][TEAMS][W][2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wave / W, tw = wave % W;
    const int lane = threadIdx.x - team * W * 64;
    int N = p.N;
    const T *X = static_cast<const T *>(p.X);
    T *Y = static_cast<T *>(p.Y);

    // elements of this wave's part of a row
    int mine = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) mine += min(max(N - P::col(tw * 64, c), 0), 64 * VE);
    const float n_w = (float)mine, rn_w = mine ? 1.0f / n_w : 0.0f;
    const bool whole = mine == C * 64 * VE;
    float w[KEEP ? C : 1][VE], b[KEEP ? C : 1][VE];
    if constexpr (KEEP) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            load_columns(w[c], p.weight, P::col(lane, c), N, whole, 1.0f);
            load_columns(b[c], p.bias, P::col(lane, c), N, whole, 0.0f);
        }
    }

    const int step = gridDim.x * TEAMS;
    int row = blockIdx.x * TEAMS + team;
    u32x4 next[C];
    auto fetch = [&](int r) {
#pragma unroll
        for (int c = 0; c < C; ++c) next[c] = load_chunk<T, W * C == 1>(X + (int64_t)r * p.ldx, P::col(lane, c), N, whole);
    };
    if (KEEP && row < p.rows) fetch(row);
    int flip = 0;
    // the workgroup's first team has a row in every pass, so that all meet at the barriers
#pragma unroll 1
    for (int first = blockIdx.x * TEAMS; first < p.rows; first += step, row += step, flip ^= 1) {
        N = renewed(p.N);
        if (!KEEP && row < p.rows) fetch(row);
        u32x4 x[C];
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = next[c];
        if (KEEP && p.rows - row > step) fetch(row + step);
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < VE; ++e) s += element<T>(x[c], e);
        float m = wave_sum(s) * rn_w, q = 0.0f;
        if (whole) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float d = element<T>(x[c], e) - m;
                    q = __builtin_fmaf(d, d, q);
                }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float d = P::col(lane, c) + e < N ? element<T>(x[c], e) - m : 0.0f;
                    q = __builtin_fmaf(d, d, q);
                }
        }
        q = wave_sum(q);
        if constexpr (W > 1) {
            if ((lane & 63) == 0) {
                slots[flip][team][tw][0] = m;
                slots[flip][team][tw][1] = q;
            }
            __syncthreads();
            float mean = 0.0f;
            int n[W];
#pragma unroll
            for (int v = 0; v < W; ++v) {
                n[v] = 0;
#pragma unroll
                for (int c = 0; c < C; ++c) n[v] += min(max(N - P::col(v * 64, c), 0), 64 * VE);
                mean = __builtin_fmaf(slots[flip][team][v][0], (float)n[v] * p.rn, mean);
            }
            q = 0.0f;
#pragma unroll
            for (int v = 0; v < W; ++v) {
                const float d = slots[flip][team][v][0] - mean;
                q += __builtin_fmaf((float)n[v] * d, d, slots[flip][team][v][1]);
            }
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
                    load_columns(wc, p.weight, P::col(lane, c) + renewed(0), N, whole, 1.0f);
                    load_columns(bc, p.bias, P::col(lane, c) + renewed(0), N, whole, 0.0f);
                }
                float y[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) y[e] = __builtin_fmaf((element<T>(x[c], e) - m) * r, wc[e], bc[e]);
                store_chunk(Y + (int64_t)row * p.ldy, P::col(lane, c), N, whole, y);
            }
            if (lane == 0) {
                if (p.mean) p.mean[row] = m;
                if (p.rstd) p.rstd[row] = r;
            }
        }
    }
}

template <class T, int W, int C, int TEAMS>
__global__ __launch_bounds__(W * 64 * TEAMS) void norm_grad(NormParams p) {
    using P = Part<T, W, C>;
    constexpr int VE = P::VE;
    constexpr bool KEEP = C <= 2;
    __shared__ float slots[2][TEAMS][W][2];
    // the column sums of the teams, one half (weight, bias) after the other
    __shared__ float sums[TEAMS > 1 ? (TEAMS - 1) * W * 64 * VE * C : 1];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wave / W, tw = wave % W;
    const int lane = threadIdx.x - team * W * 64;
    int N = p.N;
    const T *X = static_cast<const T *>(p.X), *dY = static_cast<const T *>(p.Y), *Cm = static_cast<const T *>(p.C);
    T *dX = static_cast<T *>(p.dX);

    const bool whole = P::col(tw * 64 + 64, C - 1) <= N;   // the wave's chunks all lie inside the row
    float w[KEEP ? C : 1][VE];
    if constexpr (KEEP) {
#pragma unroll
        for (int c = 0; c < C; ++c) load_columns(w[c], p.weight, P::col(lane, c), N, whole, 1.0f);
    }
    float dw[C][VE], db[C][VE];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < VE; ++e) dw[c][e] = db[c][e] = 0.0f;

    const int step = gridDim.x * TEAMS;
    int row = blockIdx.x * TEAMS + team;
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
            nx[c] = load_chunk<T, W * C == 1>(X + (int64_t)r * p.ldx, P::col(lane, c), N, whole);
            ny[c] = load_chunk<T, W * C == 1>(dY + (int64_t)r * p.ldy, P::col(lane, c), N, whole);
        }
        nm = p.mean[r];
        nr = p.rstd[r];
    };
    clear();
    if (KEEP && row < p.rows) fetch(row);
    int flip = 0;
#pragma unroll 1
    for (int first = blockIdx.x * TEAMS; first < p.rows; first += step, row += step, flip ^= 1) {
        N = renewed(p.N);
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
            for (int c = 0; c < C; ++c) res[c] = load_chunk<T, W * C == 1>(Cm + (int64_t)row * p.ldx, P::col(lane, c), N, whole);
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
            if (!KEEP) load_columns(wc, p.weight, P::col(lane, c) + renewed(0), N, whole, 1.0f);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float dy = element<T>(y[c], e), h = (element<T>(x[c], e) - m) * r, g = dy * wc[e];
                sg += g;
                sgh = __builtin_fmaf(g, h, sgh);
                dw[c][e] = __builtin_fmaf(dy, h, dw[c][e]);
                db[c][e] += dy;
            }
            chunk_done();
        }
        sg = wave_sum(sg);
        sgh = wave_sum(sgh);
        if constexpr (W > 1) {
            if ((lane & 63) == 0) {
                slots[flip][team][tw][0] = sg;
                slots[flip][team][tw][1] = sgh;
            }
            __syncthreads();
            sg = sgh = 0.0f;
#pragma unroll
            for (int v = 0; v < W; ++v) {
                sg += slots[flip][team][v][0];
                sgh += slots[flip][team][v][1];
            }
        }
        sg *= p.rn;
        sgh *= p.rn;
        if (on) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                forget(x[c]);
                forget(y[c]);
                if (!KEEP && p.has_beta) res[c] = load_chunk<T, W * C == 1>(Cm + (int64_t)row * p.ldx, P::col(lane, c), N, whole);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float (&wc)[VE] = w[KEEP ? c : 0];
                if (!KEEP) load_columns(wc, p.weight, P::col(lane, c) + renewed(0), N, whole, 1.0f);
                float d[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float dy = element<T>(y[c], e), h = (element<T>(x[c], e) - m) * r;
                    d[e] = r * (__builtin_fmaf(dy, wc[e], -sg) - h * sgh);
                    if (p.has_beta) d[e] = __builtin_fmaf(p.beta, element<T>(res[c], e), d[e]);
                }
                store_chunk(dX + (int64_t)row * p.ldx, P::col(lane, c), N, whole, d);
                chunk_done();
            }
        }
    }
    N = p.N;
    if (!p.part) return;
    // one partial sum per column and workgroup
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
        if (team == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int n = P::col(lane, c);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (n + e < N) out[half * N + n + e] = half ? db[c][e] : dw[c][e];
            }
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

template <class T, int W, int C, int TEAMS, bool GRAD>
hipError_t launch(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream) {
    if (s.teams != TEAMS) return hipErrorInvalidValue;
    if constexpr (GRAD) hipLaunchKernelGGL((norm_grad<T, W, C, TEAMS>), dim3(grid), dim3(W * 64 * TEAMS), 0, stream, p);
    else hipLaunchKernelGGL((norm_forward<T, W, C, TEAMS>), dim3(grid), dim3(W * 64 * TEAMS), 0, stream, p);
    return hipGetLastError();
}

template <class T, bool GRAD>
hipError_t by_shape(const NormParams &p, NormShape s, unsigned grid, hipStream_t stream) {
#define TGE_NORM_CASE(W, C) \
    case (W) * 8 + (C): return launch<T, W, C, norm_teams(W, GRAD), GRAD>(p, s, grid, stream)
    switch (s.waves * 8 + s.chunks) {
        TGE_NORM_CASE(1, 1);
        TGE_NORM_CASE(1, 2);
        TGE_NORM_CASE(2, 2);
        TGE_NORM_CASE(3, 2);
        TGE_NORM_CASE(4, 2);
        TGE_NORM_CASE(6, 2);
        TGE_NORM_CASE(8, 2);
        TGE_NORM_CASE(12, 2);
        TGE_NORM_CASE(16, 2);
        TGE_NORM_CASE(16, 3);
        TGE_NORM_CASE(16, 4);
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
