// Routing of rows to experts for gfx950: the choice of the k largest of each row's logits, their
// softmax weights, the per-expert counts as offsets, the rows' order by expert, the balance loss, and
// the gradient towards the logits.
//
//   p = softmax(logits of a row);  w = p of the chosen experts (over their sum with `normalize`)
//   f_e = count_e / (k T'),  loss = E sum_e f_e (mean over the T' rows in use of p_e)
//   slope_e = E f_e / T' = d loss / d p_e;  f is constant for the gradient
//   d logit_j = p_j (h_j - sum p h),  h = dloss slope (+ the chosen's dweight, or with normalize apart:
//   + w_j (dweight_j - sum w dweight) for the chosen)
//
// A row belongs to 16, 32 or 64 lanes of a wave with up to 16 consecutive experts each, so that maxima
// and sums need a few lane moves and no memory.  The choice compares logits, not probabilities: of
// equal ones the lowest expert is taken, whatever the rounding of the softmax; NaN and minus
// infinity are never chosen.  Bound: the logits' bytes for many rows, the moves of the k choices one
// after another per row, launches for few.
//
// The order is stable (by expert, then row, then choice) and has no atomics whose order shows: a
// workgroup counts its choices per expert in LDS, the counts are summed over the workgroups in order,
// and each choice's place is its expert's start + the choices of earlier workgroups and waves + its
// rank among the lanes of its wave that chose the same expert (a ballot per bit of the expert).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"

namespace tge {
namespace {

using namespace dev;

constexpr float NEG_INF = -__builtin_inff();
constexpr float ROUTE_LOG2E = 1.4426950408889634f;
constexpr int ROUTE_THREADS = 256, ROUTE_WAVES = ROUTE_THREADS / 64;

__device__ __forceinline__ float as_float(int v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ int as_int(float v) { return __builtin_bit_cast(int, v); }

// v of the lane N places on in the ring of 16 lanes (N a constant), or of the lane 16 or 32 away.
template <int N>
__device__ __forceinline__ int ring(int v) { return __builtin_amdgcn_update_dpp(0, v, 0x120 + N, 0xf, 0xf, true); }

// Reduction over a row's lanes, the result in each of them.
template <int LANES, class Op>
__device__ __forceinline__ int over_lanes(int v, Op op) {
    v = op(v, ring<8>(v));
    v = op(v, ring<4>(v));
    v = op(v, ring<2>(v));
    v = op(v, ring<1>(v));
    if constexpr (LANES >= 32) v = op(v, __builtin_amdgcn_ds_swizzle(v, 0x401f));   // lane ^ 16
    if constexpr (LANES >= 64) v = op(v, __shfl_xor(v, 32));
    return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
    return as_float(over_lanes<LANES>(as_int(v), [](int a, int b) { return as_int(__builtin_fmaxf(as_float(a), as_float(b))); }));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    return as_float(over_lanes<LANES>(as_int(v), [](int a, int b) { return as_int(as_float(a) + as_float(b)); }));
}
template <int LANES>
__device__ __forceinline__ int lanes_min(int v) {
    return over_lanes<LANES>(v, [](int a, int b) { return min(a, b); });
}

// A lane's PER consecutive logits of a row in fp32, minus infinity past the last expert.
template <class T, int PER>
__device__ __forceinline__ void load_logits(const T *row, int first, int experts, float (&x)[PER]) {
    if (first + PER <= experts) {
        T t[PER];
        __builtin_memcpy(t, row + first, sizeof(t));
#pragma unroll
        for (int v = 0; v < PER; ++v) x[v] = (float)t[v];
    } else {
#pragma unroll
        for (int v = 0; v < PER; ++v) x[v] = first + v < experts ? (float)row[first + v] : NEG_INF;
    }
}

// e^(x - m) of a lane's logits in place, and their sum over the row.  A row without a logit above minus
// infinity has no probabilities: all 0 (NaN where a logit is).
template <int LANES, int PER>
__device__ __forceinline__ float exponentials(float (&x)[PER], float m) {
    const float at = m == NEG_INF ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < PER; ++v) {
        x[v] = __builtin_amdgcn_exp2f((x[v] - at) * ROUTE_LOG2E);
        s += x[v];
    }
    return lanes_sum<LANES>(s);
}

template <int PER>
__device__ __forceinline__ float largest(const float (&x)[PER]) {
    float m = NEG_INF;
#pragma unroll
    for (int v = 0; v < PER; ++v) m = __builtin_fmaxf(m, x[v]);
    return m;
}

// Running totals of the choices: places of the workgroup's rows.  hist: LDS, a row of E counters per
// wave.  start[e]: where the workgroup's choices of expert e begin.  Choices are dealt to the waves in
// consecutive pieces.  Called by all threads of the workgroup.
__device__ void place_choices(const RouteParams &p, int row0, int rows, const int *start, int total, int *hist) {
    const int E = p.experts, n = rows * p.k;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = (n + 63) / 64, per = (chunks + ROUTE_WAVES - 1) / ROUTE_WAVES;
    const int c0 = min(wave * per, chunks), c1 = min(c0 + per, chunks);
    const int64_t base = (int64_t)row0 * p.k;
    int *mine = hist + wave * E;
    int bits = 0;
    while ((1 << bits) < E) ++bits;
    for (int i = threadIdx.x; i < ROUTE_WAVES * E; i += ROUTE_THREADS) hist[i] = 0;
    __syncthreads();
    // first the counts of every wave, then the places
    for (int pass = 0; pass < 2; ++pass) {
        for (int c = c0; c < c1; ++c) {
            const int i = c * 64 + lane;
            const int e = i < n ? p.index[base + i] : -1;
            uint64_t same = __ballot(e >= 0);
            for (int b = 0; b < bits; ++b) {
                const uint64_t set = __ballot(e >> b & 1);
                same &= e >> b & 1 ? set : ~set;
            }
            if (e >= 0) {
                const int rank = __popcll(same & ((1ull << lane) - 1)), count = __popcll(same);
                const int at = mine[e];
                // (the lanes of one expert read its counter before the first of them moves it on: one
                // wave's LDS operations execute in order)
                __builtin_amdgcn_wave_barrier();
                if (rank == 0) mine[e] = at + count;
                if (pass) {
                    const int place = at + rank;
                    p.order[place] = (int)(base + i);
                    p.place[base + i] = place;
                }
            } else if (pass && i < n) {
                p.place[base + i] = -1;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (pass && i < n && base + i >= total) p.order[base + i] = -1;
        }
        __syncthreads();
        if (pass) break;
        for (int e = threadIdx.x; e < E; e += ROUTE_THREADS) {
            int at = start[e];
#pragma unroll
            for (int w = 0; w < ROUTE_WAVES; ++w) {
                const int h = hist[w * E + e];
                hist[w * E + e] = at;
                at += h;
            }
        }
        __syncthreads();
    }
}

// Exclusive running sum of E values of LDS, in place, by the first wave; the sum in v[E].
__device__ __forceinline__ void scan_experts(int *v, int E) {
    if (threadIdx.x < 64) {
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + (int)threadIdx.x;
            const int x = e < E ? v[e] : 0, s = wave_scan_add(x);
            if (e < E) v[e] = carry + s - x;
            carry += __builtin_amdgcn_readlane(s, 63);
        }
        if (threadIdx.x == 0) v[E] = carry;
    }
    __syncthreads();
}

// Offsets, slope and loss from the totals: starts[E + 1] (LDS), used rows, summed probabilities.  In
// 64 bits: one value per expert.
__device__ void finish_totals(const RouteParams &p, const int *starts, int used, const float *ptotal, double *part) {
    const int E = p.experts;
    for (int e = threadIdx.x; e <= E; e += ROUTE_THREADS) p.offsets[e] = starts[e];
    double s = 0.0;
    const double scale = used > 0 ? (double)E / p.k / used / used : 0.0;
    for (int e = threadIdx.x; e < E; e += ROUTE_THREADS) {
        const double slope = scale * (starts[e + 1] - starts[e]);
        if (p.slope) p.slope[e] = (float)slope;
        s += slope * ptotal[e];
    }
    if (!p.loss) return;
    part[threadIdx.x] = s;
    __syncthreads();
    for (int h = ROUTE_THREADS / 2; h > 0; h /= 2) {
        if ((int)threadIdx.x < h) part[threadIdx.x] += part[threadIdx.x + h];
        __syncthreads();
    }
    if (threadIdx.x == 0) p.loss[0] = (float)part[0];
}

// ALL: one workgroup does the whole routing.
template <class T, int LANES, int PER, bool ALL>
__global__ __launch_bounds__(ROUTE_THREADS) void choose(RouteParams p) {
    constexpr int ROWS = 64 / LANES;                 // rows of a wave at a time
    constexpr int WIDTH = LANES * PER;               // experts, rounded up
    constexpr int SLOTS = ROUTE_WAVES * ROWS;
    __shared__ int hist[ALL ? ROUTE_WAVES * WIDTH : WIDTH];
    __shared__ int starts[WIDTH + 1];
    __shared__ float psum[SLOTS * WIDTH];
    __shared__ int used_rows[ROUTE_WAVES];
    const int E = p.experts, k = p.k;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = lane / LANES, l = lane % LANES, first = l * PER;
    const int row0 = blockIdx.x * p.block_rows, rows = min(p.block_rows, p.rows - row0);
    for (int e = threadIdx.x; e < WIDTH; e += ROUTE_THREADS) hist[e] = 0;
    __syncthreads();
    float ps[PER];
#pragma unroll
    for (int v = 0; v < PER; ++v) ps[v] = 0.0f;
    int used = 0;
#pragma unroll 1
    for (int r = wave * ROWS + slot; r < (rows + ROWS - 1) / ROWS * ROWS; r += SLOTS) {
        const int row = row0 + r;
        const bool on = r < rows && (!p.mask || p.mask[row]);
        float x[PER], left[PER];
        if (on) {
            load_logits(static_cast<const T *>(p.logits) + (int64_t)row * p.ldl, first, E, x);
        } else {
#pragma unroll
            for (int v = 0; v < PER; ++v) x[v] = NEG_INF;
        }
#pragma unroll
        for (int v = 0; v < PER; ++v) left[v] = x[v] == x[v] ? x[v] : NEG_INF;   // NaN is not chosen
        const float m = lanes_max<LANES>(largest(left));
        // the choices, one after another; lane j keeps the j-th
        int chosen = -1;
        float value = NEG_INF;
#pragma unroll 1
        for (int j = 0; j < k; ++j) {
            const float best = j == 0 ? m : lanes_max<LANES>(largest(left));
            int at = 1 << 30;
#pragma unroll
            for (int v = PER - 1; v >= 0; --v) at = left[v] == best ? first + v : at;
            at = lanes_min<LANES>(at);
            if (best == NEG_INF) at = -1;
#pragma unroll
            for (int v = 0; v < PER; ++v) left[v] = first + v == at ? NEG_INF : left[v];
            if (l == j) {
                chosen = at;
                value = best;
            }
        }
        const float s = exponentials<LANES>(x, m), inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
        for (int v = 0; v < PER; ++v) ps[v] = __builtin_fmaf(x[v], inv, ps[v]);
        if (m > NEG_INF && l == 0) ++used;
        float w = chosen >= 0 ? __builtin_amdgcn_exp2f((value - m) * ROUTE_LOG2E) : 0.0f;
        // NaN among the logits makes the weights NaN
        if (p.normalize) {
            const float all = lanes_sum<LANES>(w);
            w = s == s ? (chosen >= 0 ? w / all : 0.0f) : chosen >= 0 ? s : 0.0f;
        } else {
            w *= chosen >= 0 ? inv : 0.0f;
        }
        if (r < rows && l < k) {
            p.index[(int64_t)row * k + l] = chosen;
            p.weight[(int64_t)row * k + l] = w;
            if (chosen >= 0) atomicAdd(&hist[chosen], 1);   // counts: any order gives the same
        }
    }
    // probabilities: the rows' slots are added up in order
#pragma unroll
    for (int v = 0; v < PER; ++v) psum[(wave * ROWS + slot) * WIDTH + first + v] = ps[v];
    for (int h = LANES; h < 64; h *= 2) used += __shfl_xor(used, h);   // lane 0 of every row counts
    if (lane == 0) used_rows[wave] = used;
    __syncthreads();
    int all_used = 0;
#pragma unroll
    for (int w = 0; w < ROUTE_WAVES; ++w) all_used += used_rows[w];
    for (int e = threadIdx.x; e < E; e += ROUTE_THREADS) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) t += psum[i * WIDTH + e];
        if constexpr (ALL) psum[e] = t;
        else p.psum[(int64_t)blockIdx.x * E + e] = t;
        if constexpr (!ALL) p.hist[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
        if constexpr (ALL) starts[e] = hist[e];
    }
    if constexpr (!ALL) {
        if (threadIdx.x == 0) p.hist[(int64_t)blockIdx.x * (E + 1) + E] = all_used;
    } else {
        __shared__ double part[ROUTE_THREADS];
        __syncthreads();
        scan_experts(starts, E);
        finish_totals(p, starts, all_used, psum, part);
        __threadfence_block();                       // the choices written above are read again
        place_choices(p, row0, rows, starts, starts[E], hist);
    }
}

// Running sums over the workgroups, per column (expert, or used rows): hist becomes the sum of the
// workgroups before, total the sum of all; the probabilities' sums in 64 bits.  16 columns per
// workgroup, the blocks in 16 runs.
constexpr int SUM_COLS = 16, SUM_RUNS = ROUTE_THREADS / SUM_COLS;
__global__ __launch_bounds__(ROUTE_THREADS) void sum_blocks(RouteParams p) {
    __shared__ int counts[SUM_RUNS][SUM_COLS];
    __shared__ double probs[SUM_RUNS][SUM_COLS];
    const int E = p.experts, cols = E + 1;
    const int c = threadIdx.x % SUM_COLS, run = threadIdx.x / SUM_COLS, e = blockIdx.x * SUM_COLS + c;
    const int per = (p.blocks + SUM_RUNS - 1) / SUM_RUNS;
    const int b0 = min(run * per, p.blocks), b1 = min(b0 + per, p.blocks);
    int n = 0;
    double q = 0.0;
    if (e < cols) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) n += p.hist[(int64_t)b * cols + e];
    }
    if (e < E) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) q += p.psum[(int64_t)b * E + e];
    }
    counts[run][c] = n;
    probs[run][c] = q;
    __syncthreads();
    if (e >= cols) return;
    int at = 0, all = 0;
    double sum = 0.0;
    for (int r = 0; r < SUM_RUNS; ++r) {
        if (r < run) at += counts[r][c];
        all += counts[r][c];
        sum += probs[r][c];
    }
    if (run == 0) {
        p.total[e] = all;
        if (e < E) p.ptotal[e] = (float)sum;
    }
    if (e < E) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) {
            const int64_t i = (int64_t)b * cols + e;
            const int h = p.hist[i];
            p.hist[i] = at;
            at += h;
        }
    }
}

__global__ __launch_bounds__(ROUTE_THREADS) void place_blocks(RouteParams p) {
    __shared__ int hist[ROUTE_WAVES * ROUTE_MAX_EXPERTS];
    __shared__ int starts[ROUTE_MAX_EXPERTS + 1];
    __shared__ double part[ROUTE_THREADS];
    const int E = p.experts;
    for (int e = threadIdx.x; e < E; e += ROUTE_THREADS) starts[e] = p.total[e];
    __syncthreads();
    scan_experts(starts, E);
    if (blockIdx.x == 0) finish_totals(p, starts, p.total[E], p.ptotal, part);
    const int total = starts[E];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += ROUTE_THREADS) starts[e] += p.hist[(int64_t)blockIdx.x * (E + 1) + e];
    __syncthreads();
    const int row0 = blockIdx.x * p.block_rows;
    place_choices(p, row0, min(p.block_rows, p.rows - row0), starts, total, hist);
}

template <class T, int LANES, int PER>
__global__ __launch_bounds__(ROUTE_THREADS) void grad(RouteParams p) {
    constexpr int ROWS = 64 / LANES, SLOTS = ROUTE_WAVES * ROWS, WIDTH = LANES * PER;
    constexpr int NONE = -1;                         // (as a float a NaN that no arithmetic gives)
    __shared__ __attribute__((aligned(16))) int given[SLOTS][WIDTH];
    const int E = p.experts, k = p.k;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = wave * ROWS + lane / LANES, l = lane % LANES, first = l * PER;
    int *const mine = given[slot];
    float slope[PER];
    const float dloss = p.dloss && p.slope ? p.dloss[0] : 0.0f;
#pragma unroll
    for (int v = 0; v < PER; ++v) {
        slope[v] = p.dloss && p.slope && first + v < E ? dloss * p.slope[first + v] : 0.0f;
        mine[first + v] = NONE;
    }
    const int step = gridDim.x * SLOTS;
#pragma unroll 1
    for (int64_t row = (int64_t)blockIdx.x * SLOTS + slot; row - lane / LANES < p.rows; row += step) {
        const bool on = row < p.rows && (!p.mask || p.mask[row]);
        float x[PER];
        if (on) {
            load_logits(static_cast<const T *>(p.logits) + row * p.ldl, first, E, x);
        } else {
#pragma unroll
            for (int v = 0; v < PER; ++v) x[v] = NEG_INF;
        }
        // the gradient of the weights, spread to the chosen experts' lanes
        int at = -1;
        if (on && p.dweight && l < k) {
            at = p.index[row * k + l];
            if (at < 0 || at >= E) at = -1;
            else mine[at] = as_int(p.dweight[row * k + l]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        float g[PER];
        bool taken[PER];
#pragma unroll
        for (int v = 0; v < PER; ++v) {
            const int w = mine[first + v];
            taken[v] = w != NONE;
            g[v] = taken[v] ? as_float(w) : 0.0f;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (at >= 0) mine[at] = NONE;                // for the next row
        float known[PER];
#pragma unroll
        for (int v = 0; v < PER; ++v) known[v] = x[v] == x[v] ? x[v] : NEG_INF;
        const float m = lanes_max<LANES>(largest(known));
        const float s = exponentials<LANES>(x, m), inv = s == 0.0f ? 0.0f : 1.0f / s;
        float d[PER];
        if (p.normalize) {
            float sp = 0.0f, sw = 0.0f, swg = 0.0f;
#pragma unroll
            for (int v = 0; v < PER; ++v) {
                x[v] *= inv;
                sp = __builtin_fmaf(x[v], slope[v], sp);
                sw += taken[v] ? x[v] : 0.0f;
                swg = __builtin_fmaf(x[v], g[v], swg);
            }
            sp = lanes_sum<LANES>(sp);
            sw = lanes_sum<LANES>(sw);
            swg = lanes_sum<LANES>(swg);
            const float over = sw == 0.0f ? 0.0f : 1.0f / sw, mean = swg * over;
#pragma unroll
            for (int v = 0; v < PER; ++v) d[v] = x[v] * (slope[v] - sp + (taken[v] ? over * (g[v] - mean) : 0.0f));
        } else {
            float sp = 0.0f;
#pragma unroll
            for (int v = 0; v < PER; ++v) {
                x[v] *= inv;
                g[v] += slope[v];
                sp = __builtin_fmaf(x[v], g[v], sp);
            }
            sp = lanes_sum<LANES>(sp);
#pragma unroll
            for (int v = 0; v < PER; ++v) d[v] = x[v] * (g[v] - sp);
        }
        if (row < p.rows) {
            T *out = static_cast<T *>(p.dlogits) + row * p.ldl + first;
            T t[PER];
#pragma unroll
            for (int v = 0; v < PER; ++v) t[v] = (T)(on ? d[v] : 0.0f);   // left out: 0, whatever dloss is
            if (first + PER <= E) {
                __builtin_memcpy(out, t, sizeof(t));
            } else {
#pragma unroll
                for (int v = 0; v < PER; ++v)
                    if (first + v < E) out[v] = t[v];
            }
        }
    }
}

template <class T, int LANES, int PER>
hipError_t launch_choose(const RouteParams &p, hipStream_t s) {
    if (p.blocks == 1) hipLaunchKernelGGL((choose<T, LANES, PER, true>), dim3(1), dim3(ROUTE_THREADS), 0, s, p);
    else hipLaunchKernelGGL((choose<T, LANES, PER, false>), dim3(p.blocks), dim3(ROUTE_THREADS), 0, s, p);
    return hipGetLastError();
}
template <class T, int LANES, int PER>
hipError_t launch_grad(const RouteParams &p, unsigned grid, hipStream_t s) {
    hipLaunchKernelGGL((grad<T, LANES, PER>), dim3(grid), dim3(ROUTE_THREADS), 0, s, p);
    return hipGetLastError();
}

template <class T, bool GRAD>
hipError_t by_shape(const RouteParams &p, RouteShape s, unsigned grid, hipStream_t stream) {
#define TGE_ROUTE_CASE(L, P)                                                     \
    case (L) * 32 + (P):                                                         \
        if constexpr (GRAD) return launch_grad<T, L, P>(p, grid, stream);        \
        else return launch_choose<T, L, P>(p, stream)
    switch (s.lanes * 32 + s.per) {
        TGE_ROUTE_CASE(16, 1);
        TGE_ROUTE_CASE(16, 2);
        TGE_ROUTE_CASE(16, 4);
        TGE_ROUTE_CASE(16, 8);
        TGE_ROUTE_CASE(32, 8);
        TGE_ROUTE_CASE(64, 8);
        TGE_ROUTE_CASE(64, 16);
    default: return hipErrorInvalidValue;
    }
#undef TGE_ROUTE_CASE
}

}  // namespace

#if defined(TGE_TYPE_F32)
hipError_t route_choose_f32(const RouteParams &p, RouteShape s, hipStream_t st) { return by_shape<float, false>(p, s, 0, st); }
hipError_t route_grad_f32(const RouteParams &p, RouteShape s, unsigned g, hipStream_t st) { return by_shape<float, true>(p, s, g, st); }

hipError_t route_place(const RouteParams &p, hipStream_t stream) {
    hipLaunchKernelGGL(sum_blocks, dim3((p.experts + SUM_COLS) / SUM_COLS), dim3(ROUTE_THREADS), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(place_blocks, dim3(p.blocks), dim3(ROUTE_THREADS), 0, stream, p);
    return hipGetLastError();
}
#elif defined(TGE_TYPE_F16)
hipError_t route_choose_f16(const RouteParams &p, RouteShape s, hipStream_t st) { return by_shape<_Float16, false>(p, s, 0, st); }
hipError_t route_grad_f16(const RouteParams &p, RouteShape s, unsigned g, hipStream_t st) { return by_shape<_Float16, true>(p, s, g, st); }
#elif defined(TGE_TYPE_BF16)
hipError_t route_choose_bf16(const RouteParams &p, RouteShape s, hipStream_t st) { return by_shape<__bf16, false>(p, s, 0, st); }
hipError_t route_grad_bf16(const RouteParams &p, RouteShape s, unsigned g, hipStream_t st) { return by_shape<__bf16, true>(p, s, g, st); }
#else
#error "define one TGE_TYPE_* macro"
#endif

}  // namespace tge
