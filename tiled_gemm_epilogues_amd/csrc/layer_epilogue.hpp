// The epilogue of a layer's products: D = act(z) + beta * C with z = alpha * acc + bias, z kept on
// request, or, for the gradient, D = act'(Z) * alpha * acc.  Included by the kernels' layer instances.
//
// Activations, in fp32 on the accumulator's value:
//   silu        z s(z), s(w) = 1 / (1 + e^-w)
//   gelu_tanh   z s(w), w = z (a + b z^2), a = 2 sqrt(2/pi), b = 0.044715 a: (1 + tanh u) / 2 = s(2u)
//   gelu        z Phi(z).  With x = |z|, 1 - Phi(x) = e^(-x^2/2) R(x): R falls from 1/2 like 1 / x, and
//               is approximated by a polynomial in t = 1 / (1 + p x) without a constant term, fitted to
//               it on [0, 14] for the smallest relative error by linear programming: degree 6, 8.3e-6
//               (16-bit results: a sixtieth of fp16's half step), degree 9, 8.4e-8 (fp32 results; with
//               its coefficients in fp32).
//               Relative, so that the negative tail keeps its digits.
// Their slopes: s + z dw/dz s (1 - s), and Phi(z) + z e^(-z^2/2) / sqrt(2 pi).
// Cycles per value and wave (16 lanes; exponential and reciprocal take four times as long): silu and
// gelu_tanh some 50, gelu 80.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"

namespace tge {
namespace dev {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float TANH_A = 1.5957691216057308f, TANH_B = 0.07135481627159852f;
constexpr float SQRT_2PI_INV = 0.3989422804014327f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

// s(w) from v = -w log2(e).
__device__ __forceinline__ float logistic(float v) { return rcp_fast(1.0f + exp2_fast(v)); }

// s + z g s (1 - s) from v = -w log2(e), g = dw/dz.  With t = e^-|w| and d = 1 / (1 + t), s is d h, h 1 or t by
// the side that w is on, and s (1 - s) is t d^2 (the difference would have no digits left where s is near 1,
// and z g is large there).  t goes to 0 on both sides, and z t is taken before g, which is finite: at large z, where w
// and z g pass fp32's range, the slope is 0 or 1.  t below 2^-126 is 0: an error of 3e-36 at most.  (8192 x 16384 x
// 4096 with gelu_tanh 900 us; taken from z g, which is wrong at large z, 896; with K 256 186 and 181.)
__device__ __forceinline__ float logistic_slope(float z, float g, float v) {
    const float t = exp2_fast(-__builtin_fabsf(v)), d = rcp_fast(1.0f + t), h = v > 0.0f ? t : 1.0f;
    return d * __builtin_fmaf(z * t * g, d, h);
}

// e^(-z^2/2), and Phi(z) from it.
__device__ __forceinline__ float gauss(float z) { return exp2_fast(z * z * (-0.5f * LOG2E)); }
template <int ES>
__device__ __forceinline__ float phi(float z, float e) {
    const float x = __builtin_fabsf(z);
    float r;
    if constexpr (ES == 2) {
        const float t = rcp_fast(__builtin_fmaf(0.30f, x, 1.0f));
        r = __builtin_fmaf(-0.07709785550832748f, t, 0.21603821218013763f);
        r = __builtin_fmaf(r, t, -0.016949163749814034f);
        r = __builtin_fmaf(r, t, 0.14419682323932648f);
        r = __builtin_fmaf(r, t, 0.11374185234308243f);
        r = __builtin_fmaf(r, t, 0.12007423490285873f) * t;
    } else {
        const float t = rcp_fast(__builtin_fmaf(0.26f, x, 1.0f));
        r = __builtin_fmaf(0.030811583623290062f, t, -0.15416397154331207f);
        r = __builtin_fmaf(r, t, 0.25390198826789856f);
        r = __builtin_fmaf(r, t, -0.15327833592891693f);
        r = __builtin_fmaf(r, t, 0.16224147379398346f);
        r = __builtin_fmaf(r, t, 0.05061749741435051f);
        r = __builtin_fmaf(r, t, 0.1030985414981842f);
        r = __builtin_fmaf(r, t, 0.10301216691732407f);
        r = __builtin_fmaf(r, t, 0.10375905781984329f) * t;
    }
    const float q = e * r;               // the far side's share
    return z < 0.0f ? q : 1.0f - q;
}

// act(z); ES: bytes of the output's type.
template <int ACT, int ES>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == ACT_RELU) return z < 0.0f ? 0.0f : z;   // NaN stays
    if constexpr (ACT == ACT_SILU) return z * logistic(z * -LOG2E);
    if constexpr (ACT == ACT_GELU_TANH)
        return z * logistic(z * __builtin_fmaf(z * z, -LOG2E * TANH_B, -LOG2E * TANH_A));
    if constexpr (ACT == ACT_GELU) return z * phi<ES>(z, gauss(z));
    return z;
}
// act'(z)
template <int ACT, int ES>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == ACT_SILU) return logistic_slope(z, 1.0f, z * -LOG2E);
    if constexpr (ACT == ACT_GELU_TANH) {
        // (from 16 on t is 0, whatever z^2 is; NaN and infinities come with z)
        const float z2 = __builtin_fminf(z * z, 256.0f);
        return logistic_slope(z, __builtin_fmaf(z2, 3.0f * TANH_B, TANH_A),
                              z * __builtin_fmaf(z2, -LOG2E * TANH_B, -LOG2E * TANH_A));
    }
    if constexpr (ACT == ACT_GELU) {
        const float e = gauss(z);
        return __builtin_fmaf(z * e, SQRT_2PI_INV, phi<ES>(z, e));
    }
    return 1.0f;
}

// Orders this wave's LDS accesses (they execute in order; no instruction).
__device__ __forceinline__ void staging_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// f(ACT) with the launch's activation as a constant (uniform branches).
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
    case ACT_RELU: f(std::integral_constant<int, ACT_RELU>()); break;
    case ACT_SILU: f(std::integral_constant<int, ACT_SILU>()); break;
    case ACT_GELU_TANH: f(std::integral_constant<int, ACT_GELU_TANH>()); break;
    case ACT_GELU: f(std::integral_constant<int, ACT_GELU>()); break;
    default: f(std::integral_constant<int, ACT_NONE>()); break;
    }
}

// n values of one row and consecutive columns: in v alpha * acc + bias (forward) or alpha * acc, out
// the values of D; x: the values of C or, for the gradient, of Z.
template <int N, int ES, class T>
__device__ __forceinline__ void finish_values(const LayerParams &p, float (&v)[N], const T (&x)[N]) {
    if (p.grad) {
        with_act(p.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] *= act_slope<act.value, ES>((float)x[e]);
        });
        return;
    }
    with_act(p.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = act_value<act.value, ES>(v[e]);
    });
    if (p.has_beta) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = __builtin_fmaf(p.beta, (float)x[e], v[e]);
    }
}

// Rounds N values to the output type (nearest, ties to even), two at a time.
template <int N, class T>
__device__ __forceinline__ void round_values(const float (&v)[N], T (&out)[N]) {
    if constexpr (sizeof(T) == 2 && N % 2 == 0) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef T t2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int e = 0; e < N; e += 2) {
            const t2 r = __builtin_convertvector((f32x2){v[e], v[e + 1]}, t2);
            out[e] = r[0];
            out[e + 1] = r[1];
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) out[e] = (T)v[e];
    }
}

// Epilogue of a wave's 32x32 MFMA tiles (the general kernel; the accumulators' lane map is that of
// store_tile): lane l holds 4 consecutive columns of row l % 32 per register group.
template <class O, class AccV, int TM, int TN>
__device__ __forceinline__ void store_layer_tile(const LayerParams &p, int mbase, int nbase, int lane,
                                                 AccV (&acc)[TM][TN]) {
    using T = typename O::T;
    constexpr int ES = sizeof(T);
    const int hi = lane >> 5, rl = lane & 31, N = p.N;
    const float *bias = static_cast<const float *>(p.bias);
    const T *X = static_cast<const T *>(p.grad ? p.Z : p.C);
    T *D = static_cast<T *>(p.D), *Z = static_cast<T *>(p.Z);
    const bool reads = p.grad || p.has_beta;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = mbase + 32 * i + rl;
        if (m >= p.M) continue;
        const int64_t row = (int64_t)m * p.ldc;
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int n = nbase + 32 * j + 8 * g + 4 * hi;
                if (n >= N) continue;
                const int have = min(N - n, 4);
                float v[4];
                T x[4], out[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // columns past N take the last one's; they are not stored
                    const int c = n + min(e, have - 1);
                    v[e] = p.alpha * acc[i][j][4 * g + e] + (p.has_bias ? bias[c] : 0.0f);
                    x[e] = reads ? X[row + c] : (T)0;
                }
                if (!p.grad && Z) {
                    round_values(v, out);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < have) Z[row + n + e] = out[e];
                }
                finish_values<4, ES>(p, v, x);
                round_values(v, out);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < have) D[row + n + e] = out[e];
            }
    }
}

// Epilogue of a wave's 16x16 MFMA tiles (the fast kernel): NF x NF of them, WT = 16 NF rows and
// columns, in blocks of 32 rows that go through the wave's staging buffer in fp32 and come back as
// 16-byte row pieces of the output type, a lane's pieces all in the same columns.  So C and Z are
// read and written in whole lines (read in the accumulators' layout, 8 bytes of 16 rows at a time,
// the gradient of 16384 rows by 16 experts of 8192 x 2048 took 603 us where the same product
// without it takes 492; so it takes 523 to 563 by the activation, 463 without), the bias is 4 or 8
// values per lane, and the loop over the blocks is rolled
// around one copy of the activations' code (unrolled for every block it would not fit the
// instruction cache); only the step from the accumulators, whose registers must be constants, is
// there once per block.  C (Z) of the next block is loaded before the stores of this one, which it
// would wait behind.
//   staged row r: 16-byte chunk c at slot(c) ^ r, slot(c) = c for fp32 outputs; for 16-bit ones a
//   piece is the chunks 2q and 2q + 1, and even chunks stand in the row's first half, odd ones in the
//   second, so that lanes side by side read chunks side by side.
template <class O, int WT>
struct LayerStage {
    static constexpr int ES = sizeof(typename O::T);
    static constexpr int VE = 16 / ES;               // columns of a piece
    static constexpr int CH = WT / 4;                // chunks of a staged row
    static constexpr int PPR = WT / VE;              // pieces of a row
    static constexpr int NP = 32 * PPR / 64;         // pieces of a lane and block
    static constexpr int RPP = 64 / PPR;             // rows between them
    static constexpr int BYTES = 32 * WT * 4;
    __device__ __forceinline__ static int at(int r, int c) {
        constexpr int H = ES == 2 ? CH / 2 : CH;     // chunks per part
        const int part = ES == 2 ? c & 1 : 0, k = ES == 2 ? c >> 1 : c;
        return r * WT * 4 + ((part * H + (k ^ (r & (H - 1)))) << 4);
    }
};

template <class O, bool FULL, class AccV, int NF>
__device__ __forceinline__ void store_layer_staged(const LayerParams &p, int mbase, int nbase, int lane,
                                                   AccV (&acc)[NF][NF], uint8_t *stg) {
    using T = typename O::T;
    constexpr int WT = NF * 16, NB = WT / 32;
    using S = LayerStage<O, WT>;
    constexpr int VE = S::VE, NP = S::NP, ES = S::ES;
    const int M = p.M, N = p.N;
    const int n = nbase + (lane % S::PPR) * VE, r0 = lane / S::PPR;   // this lane's columns, first row
    const T *X = static_cast<const T *>(p.grad ? p.Z : p.C);
    T *D = static_cast<T *>(p.D), *Z = p.grad ? nullptr : static_cast<T *>(p.Z);
    const bool reads = p.grad || p.has_beta;
    const int have = FULL ? VE : min(max(N - n, 0), VE);              // columns inside the matrix
    typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));
    // streaming stores as in the other epilogue, by the same rule
    const bool stream_d = p.stream && FULL;

    float bv[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e)
        bv[e] = p.has_bias && e < have ? static_cast<const float *>(p.bias)[n + e] : 0.0f;

    struct Piece { T v[VE]; };
    auto load = [&](int b, int q) {
        Piece x;
        const int m = mbase + 32 * b + r0 + q * S::RPP;
        const T *src = X + (int64_t)m * p.ldc + n;
        if constexpr (FULL) {
            __builtin_memcpy(x.v, src, 16);
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e) x.v[e] = (T)0;
            if (m < M && have == VE) {
                __builtin_memcpy(x.v, src, 16);
            } else if (m < M && have > 0) {
                // past the edge the row's last value again: every load is unconditional
#pragma unroll
                for (int e = 0; e < VE; ++e) x.v[e] = src[min(e, have - 1)];
            }
        }
        return x;
    };
    auto store = [&](T *out, int b, int q, const Piece &x) {
        const int m = mbase + 32 * b + r0 + q * S::RPP;
        T *dst = out + (int64_t)m * p.ldc + n;
        u32x4 w;
        __builtin_memcpy(&w, x.v, 16);
        if constexpr (FULL) {
            if (stream_d) __builtin_nontemporal_store((u32x4u)w, reinterpret_cast<u32x4u *>(dst));
            else __builtin_memcpy(dst, &w, 16);
        } else if (m < M) {
            if (have == VE) {
                __builtin_memcpy(dst, &w, 16);
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (e < have) dst[e] = x.v[e];
            }
        }
    };

    Piece cur[NP], next[NP];
#pragma unroll
    for (int q = 0; q < NP; ++q) next[q] = Piece{};
    if (reads) {
#pragma unroll
        for (int q = 0; q < NP; ++q) next[q] = load(0, q);
    }
#pragma unroll 1
    for (int b = 0; b < NB; ++b) {
        // block b of the accumulators, row-major in the staging buffer
        staging_order();
        auto stage = [&](auto block) {
            constexpr int B = block.value;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    *reinterpret_cast<AccV *>(stg + S::at(16 * i + (lane & 15), 4 * j + (lane >> 4))) = acc[2 * B + i][j];
        };
        if constexpr (NB == 4) {
            switch (b) {
            case 0: stage(std::integral_constant<int, 0>()); break;
            case 1: stage(std::integral_constant<int, 1>()); break;
            case 2: stage(std::integral_constant<int, 2>()); break;
            default: stage(std::integral_constant<int, 3>()); break;
            }
        } else if constexpr (NB == 2) {
            if (b == 0) stage(std::integral_constant<int, 0>());
            else stage(std::integral_constant<int, 1>());
        } else {
            stage(std::integral_constant<int, 0>());
        }
#pragma unroll
        for (int q = 0; q < NP; ++q) cur[q] = next[q];
        if (reads && b + 1 < NB) {
#pragma unroll
            for (int q = 0; q < NP; ++q) next[q] = load(b + 1, q);
        }
        staging_order();
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const int r = r0 + q * S::RPP;
            float v[VE];
#pragma unroll
            for (int h = 0; h < VE / 4; ++h) {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(stg + S::at(r, (lane % S::PPR) * (VE / 4) + h));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * h + e] = __builtin_fmaf(p.alpha, a[e], bv[4 * h + e]);
            }
            Piece out;
            if (Z) {
                round_values(v, out.v);
                store(Z, b, q, out);
            }
            finish_values<VE, ES>(p, v, cur[q].v);
            round_values(v, out.v);
            store(D, b, q, out);
        }
    }
}

}  // namespace dev
}  // namespace tge
