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
// A row belongs to 16, 32 or 64 lanes of a wave with up to 16 experts each, so that maxima
// and sums need a few lane moves and no memory.  The choice compares logits, not probabilities: of
// equal ones the lowest expert is taken, whatever the rounding of the softmax; NaN and minus
// infinity are never chosen.  Bound: the logits' bytes for many rows, the moves of the k choices one
// after another per row, launches for few.
//
// The order is stable (by expert, then row, then choice) and has no atomics whose order shows: a
// workgroup counts its choices per expert in LDS, and each choice's place is its expert's start + the
// choices of earlier workgroups and waves + its rank among the lanes of its wave that chose the same
// expert (a ballot per bit of the expert).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_internal.h"

namespace tge {
namespace {

using namespace dev;

constexpr float NEG_INF = -__builtin_inff();
constexpr float ROUTE_LOG2E = 1.4426950408889634f;
constexpr int ROUTE_THREADS = 256, ROUTE_WAVES = ROUTE_THREADS / 64;   // of the gradient

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

// The experts of a lane: PER in all, whole 16-byte chunks of the row's logits side by side with the
// other lanes' (32 bytes to a lane would take every line in two accesses: the gradient of 65536 rows of
// 128 fp32 logits 21.4 us so), the v-th of them
template <class T, int LANES, int PER>
struct Share {
    static constexpr int CHUNK = 16 / (int)sizeof(T) < PER ? 16 / (int)sizeof(T) : PER;
    __device__ __forceinline__ static int expert(int l, int v) { return (v / CHUNK * LANES + l) * CHUNK + v % CHUNK; }

    // its logits in fp32, minus infinity past the last expert
    __device__ __forceinline__ static void load(const T *row, int l, int experts, float (&x)[PER]) {
#pragma unroll
        for (int c = 0; c < PER; c += CHUNK) {
            const int first = expert(l, c);
            if (first + CHUNK <= experts) {
                T t[CHUNK];
                __builtin_memcpy(t, row + first, sizeof(t));
#pragma unroll
                for (int v = 0; v < CHUNK; ++v) x[c + v] = (float)t[v];
            } else {
#pragma unroll
                for (int v = 0; v < CHUNK; ++v) x[c + v] = first + v < experts ? (float)row[first + v] : NEG_INF;
            }
        }
    }
    __device__ __forceinline__ static void store(T *row, int l, int experts, const float (&x)[PER]) {
#pragma unroll
        for (int c = 0; c < PER; c += CHUNK) {
            const int first = expert(l, c);
            T t[CHUNK];
#pragma unroll
            for (int v = 0; v < CHUNK; ++v) t[v] = (T)x[c + v];
            if (first + CHUNK <= experts) {
                __builtin_memcpy(row + first, t, sizeof(t));
            } else {
#pragma unroll
                for (int v = 0; v < CHUNK; ++v)
                    if (first + v < experts) row[first + v] = t[v];
            }
        }
    }
};

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

// A logit as a number of 32 bits whose order is that of the logits (+0 and -0 are equal; NaN counts as
// minus infinity).  Logits that may be chosen have LOWEST and more.
constexpr uint32_t LOWEST = 0x00800000u;
__device__ __forceinline__ uint32_t rank_of(float x) {
    const int b = __builtin_bit_cast(int, __builtin_fmaxf(x + 0.0f, NEG_INF));
    return (uint32_t)(b ^ (b >> 31 | (int)0x80000000));
}

// Sorts a lane's keys, the largest first: Batcher's odd-even merge network.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&v)[N]) {
    auto swap = [&](int a, int b) {
        const uint32_t hi = max(v[a], v[b]), lo = min(v[a], v[b]);
        v[a] = hi;
        v[b] = lo;
    };
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) swap(i + j, i + j + q);
}

// The choices of a wave's piece, 64 of them in each of up to AHEAD chunks that are loaded at once.  As
// many waves take part as there are rows of counters for.  index: the workgroup's choices, in memory
// or (KEPT) in LDS.
constexpr int AHEAD = 4;
template <bool KEPT>
struct Choices {
    const int32_t *index;
    int n, c0, c1;           // its choices; the wave's chunks
    int waves;               // that take part
    int held[AHEAD];

    __device__ __forceinline__ void init(const RouteParams &p, const int32_t *from, int rows, int counters) {
        index = from;
        n = rows * p.k;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        waves = min((int)blockDim.x / 64, counters / p.experts);
        const int chunks = (n + 63) / 64, per = (chunks + waves - 1) / waves;
        c0 = min(wave * per, chunks);
        c1 = min(c0 + per, chunks);
        load(c0);
    }
    __device__ __forceinline__ void load(int c) {
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int i = (c + a) * 64 + (int)(threadIdx.x & 63);
            held[a] = -1;
            if (c + a < c1 && i < n) {
                if constexpr (KEPT) held[a] = ((const __attribute__((address_space(3))) int32_t *)index)[i];
                else held[a] = index[i];
            }
        }
    }
    // f(choice's number in the workgroup, expert or -1) for every chunk of the wave
    template <class F>
    __device__ __forceinline__ void each(F f) {
        for (int c = c0; c < c1; c += AHEAD) {
            if (c1 - c0 > AHEAD) load(c);                // (else they are held from the start)
#pragma unroll
            for (int a = 0; a < AHEAD; ++a)
                if (c + a < c1) f((c + a) * 64 + (int)(threadIdx.x & 63), held[a]);
        }
    }
};

// The places of a workgroup's choices.  hist: LDS, a row of E counters per wave.  start[e]: where its
// choices of expert e begin.  Choices are dealt to the waves in consecutive pieces; the places of a
// wave's piece follow from its counts and those of the waves before.  Called by all its threads.
template <bool KEPT>
__device__ void place_choices(const RouteParams &p, int row0, Choices<KEPT> &mine, const int *start, int total, int *hist) {
    const int64_t base = (int64_t)row0 * p.k;
    const int E = p.experts, waves = mine.waves;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int *counters = hist + wave * E;                     // (a wave without one has no choices)
    int bits = 0;
    while ((1 << bits) < E) ++bits;
    for (int i = threadIdx.x; i < waves * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    mine.each([&](int, int e) {
        if (e >= 0) atomicAdd(&counters[e], 1);          // counts: any order gives the same
    });
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int at = start[e];
#pragma unroll 8
        for (int w = 0; w < waves; ++w) {
            const int h = hist[w * E + e];
            hist[w * E + e] = at;
            at += h;
        }
    }
    __syncthreads();
    mine.each([&](int i, int e) {
        uint64_t same = __ballot(e >= 0);                // lanes with this lane's expert
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot(e >> b & 1);
            same &= e >> b & 1 ? set : ~set;
        }
        if (e >= 0) {
            const int rank = __popcll(same & ((1ull << lane) - 1)), at = counters[e];
            // (the lanes of one expert read its counter before the first of them moves it on: a wave's
            // LDS operations execute in order)
            __builtin_amdgcn_wave_barrier();
            if (rank == 0) counters[e] = at + __popcll(same);
            p.order[at + rank] = (int)(base + i);
            p.place[base + i] = at + rank;
        } else if (i < mine.n) {
            p.place[base + i] = -1;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (i < mine.n && base + i >= total) p.order[base + i] = -1;
    });
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

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int h = 32; h > 0; h /= 2) v += __shfl_xor(v, h);
    return v;
}

// Offsets, slope and loss from the totals: starts[E + 1] and the probabilities' sums (LDS), the used
// rows.  In 64 bits: one value per expert.
__device__ void finish_totals(const RouteParams &p, const int *starts, int used, const float *ptotal) {
    const int E = p.experts;
    for (int e = threadIdx.x; e <= E; e += blockDim.x) p.offsets[e] = starts[e];
    const double scale = used > 0 ? (double)E / p.k / used / used : 0.0;
    if (p.slope)
        for (int e = threadIdx.x; e < E; e += blockDim.x) p.slope[e] = (float)(scale * (starts[e + 1] - starts[e]));
    if (p.loss && threadIdx.x < 64) {
        double s = 0.0;
        for (int e = threadIdx.x; e < E; e += 64) s += scale * (starts[e + 1] - starts[e]) * ptotal[e];
        s = wave_sum64(s);
        if (threadIdx.x == 0) p.loss[0] = (float)s;
    }
}

// The key of the same place in the lane 8, 4, 2 or 1 on in the ring of 16 lanes, or 16 or 32 away.
template <int STEP>
__device__ __forceinline__ uint32_t key_from(uint32_t v) {
    if constexpr (STEP <= 8) return (uint32_t)ring<STEP>((int)v);
    else if constexpr (STEP == 16) return (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x401f);
    else return (uint32_t)__shfl_xor((int)v, 32);
}

// One step of a row's choice: of the sorted keys of two lanes the LEN largest, sorted, in both.  The
// larger of the one's i-th and the other's last-but-i-th are the largest; they rise and fall once, and
// halving exchanges sort them.
template <int STEP, int LEN>
__device__ __forceinline__ void merge_lanes(uint32_t (&v)[LEN]) {
    uint32_t other[LEN];
#pragma unroll
    for (int i = 0; i < LEN; ++i) other[i] = key_from<STEP>(v[LEN - 1 - i]);
#pragma unroll
    for (int i = 0; i < LEN; ++i) v[i] = max(v[i], other[i]);
#pragma unroll
    for (int q = LEN / 2; q >= 1; q /= 2)
#pragma unroll
        for (int i = 0; i < LEN; ++i)
            if (!(i & q)) {
                const uint32_t hi = max(v[i], v[i + q]), lo = min(v[i], v[i + q]);
                v[i] = hi;
                v[i + q] = lo;
            }
}

// The k <= LEN largest keys of a row, lane j's result the j-th; keys: the lane's own, sorted.  unsure:
// (uniform) whether keys may be in the wrong order, see choose_experts.
template <int LANES, int PER, int LEN, bool EXACT>
__device__ __forceinline__ uint32_t largest_keys(const uint32_t (&key)[PER], int l, int k, bool &unsure) {
    constexpr uint32_t LAST = LANES * PER - 1;
    uint32_t v[LEN];
#pragma unroll
    for (int i = 0; i < LEN; ++i) v[i] = i < PER ? key[i < PER ? i : 0] : 0u;
    merge_lanes<8>(v);
    merge_lanes<4>(v);
    merge_lanes<2>(v);
    merge_lanes<1>(v);
    if constexpr (LANES >= 32) merge_lanes<16>(v);
    if constexpr (LANES >= 64) merge_lanes<32>(v);
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < LEN; ++j) mine = l == j ? v[j] : mine;
    if (l >= k) mine = 0;
    if constexpr (!EXACT) {
        // two neighbours of the order with the same bits left
        const uint32_t next = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, 0x101, 0xf, 0xf, true);   // lane j + 1's
        const bool bad = next >= LOWEST && (next ^ mine) <= LAST;
        // or more keys with the last one's bits, or above, than were chosen.  No row has fewer, so the
        // numbers over the wave are equal only if they are in every row
        uint32_t kth = v[0];
#pragma unroll
        for (int j = 1; j < LEN; ++j) kth = j < k ? v[j] : kth;
        const uint32_t from = max(kth & ~LAST, LOWEST);
        int above = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) above += __popcll(__ballot(key[i] >= from));
        unsure = __ballot(bad) != 0 || above != __popcll(__ballot(mine >= LOWEST));
    } else {
        unsure = false;
    }
    return mine;
}

// Choice of the j-th largest logits, j < k, of the rows of a wave; on return lane j of a row holds the j-th
// expert (-1: none is left).  A lane's logits become keys of 32 bits, their rank with its last bits
// replaced by the expert, lowest last, so that one unsigned comparison orders values and experts and no
// two keys are equal; each lane sorts its own, then lanes merge theirs in pairs (some 35 instructions a
// step, where taking one maximum after another costs as many for each choice: 65536 rows of 128, 8
// chosen, 23 us so).  16-bit logits lose nothing in the key.  fp32 logits lose their last
// bits: where two keys in order have the same bits left (the first not chosen included) it may be wrong or
// a tie, and the wave chooses again from the logits themselves.  For random logits that is about one
// row in a thousand.
template <class T, int LANES, int PER>
__device__ __forceinline__ int choose_experts(const float (&x)[PER], int l, int k) {
    using S = Share<T, LANES, PER>;
    constexpr bool EXACT = sizeof(T) == 2;
    constexpr uint32_t LAST = LANES * PER - 1;
    uint32_t key[PER];
#pragma unroll
    for (int v = 0; v < PER; ++v) key[v] = (rank_of(x[v]) & ~LAST) | (LAST - S::expert(l, v));
    sort_keys(key);
    bool unsure;
    const uint32_t taken = k <= 8 ? largest_keys<LANES, PER, 8, EXACT>(key, l, k, unsure)
                                  : largest_keys<LANES, PER, ROUTE_MAX_K, EXACT>(key, l, k, unsure);
    int chosen = taken >= LOWEST ? (int)(LAST - (taken & LAST)) : -1;
    if (!EXACT && unsure) {
        float left[PER];
#pragma unroll
        for (int v = 0; v < PER; ++v) left[v] = x[v] == x[v] ? x[v] : NEG_INF;
#pragma unroll 1
        for (int j = 0; j < k; ++j) {
            const float best = lanes_max<LANES>(largest(left));
            int at = 1 << 30;
#pragma unroll
            for (int v = PER - 1; v >= 0; --v) at = left[v] == best ? S::expert(l, v) : at;
            at = lanes_min<LANES>(at);
            if (best == NEG_INF) at = -1;
#pragma unroll
            for (int v = 0; v < PER; ++v) left[v] = S::expert(l, v) == at ? NEG_INF : left[v];
            chosen = l == j ? at : chosen;
        }
    }
    return chosen;
}

// ALL: one workgroup does the whole routing.
template <class T, int LANES, int PER, bool ALL>
__global__ __launch_bounds__(route_waves(LANES *PER) * 64) void choose(RouteParams p) {
    constexpr int ROWS = 64 / LANES;                 // rows of a wave at a time
    constexpr int WIDTH = LANES * PER;               // experts, rounded up
    constexpr int WAVES = route_waves(WIDTH), THREADS = WAVES * 64, SLOTS = WAVES * ROWS;
    __shared__ int counts[WIDTH];
    __shared__ int starts[WIDTH + 1];
    __shared__ float ptotal[WIDTH];
    // the rows at work, then the waves' summed probabilities, then their counters
    __shared__ __attribute__((aligned(16))) int shared[SLOTS * WIDTH];
    __shared__ int used_rows[WAVES];
    __shared__ int kept[ALL ? route_one_rows(WAVES, LANES) * ROUTE_MAX_K : 1];   // the choices, for their places
    const int E = p.experts, k = p.k;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    using S = Share<T, LANES, PER>;
    const int slot = lane / LANES, l = lane % LANES;
    const int row0 = blockIdx.x * p.block_rows, rows = min(p.block_rows, p.rows - row0);
    const T *logits = static_cast<const T *>(p.logits) + (int64_t)row0 * p.ldl;
    float *const psum = reinterpret_cast<float *>(shared), *const values = psum + (wave * ROWS + slot) * WIDTH;
    for (int e = threadIdx.x; e < WIDTH; e += THREADS) counts[e] = 0;
    __syncthreads();
    float ps[PER], next[PER];
#pragma unroll
    for (int v = 0; v < PER; ++v) ps[v] = 0.0f;
    int used = 0;
    int next_on = 0;
    // (loads side by side, none waiting for another)
    auto fetch = [&](int r) {
        next_on = r < rows;
        if (r < rows) {
            if (p.mask) next_on = p.mask[row0 + r];
            S::load(logits + (int64_t)r * p.ldl, l, E, next);
        }
    };
    const int end = (rows + ROWS - 1) / ROWS * ROWS; // (a wave's rows stay together)
    fetch(wave * ROWS + slot);
#pragma unroll 1
    for (int r = wave * ROWS + slot; r < end; r += SLOTS) {
        const int64_t row = row0 + r;
        float x[PER];
#pragma unroll
        for (int v = 0; v < PER; ++v) x[v] = next_on ? next[v] : NEG_INF;
        if (end - r > SLOTS) fetch(r + SLOTS);
        // the row in LDS, where its lanes find the chosen logits
#pragma unroll
        for (int v = 0; v < PER; ++v) values[S::expert(l, v)] = x[v];
        const int chosen = choose_experts<T, LANES, PER>(x, l, k);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float value = chosen >= 0 ? values[chosen] : 0.0f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float m = lanes_max<LANES>(largest(x));
        const float s = exponentials<LANES>(x, m), inv = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
#pragma unroll
        for (int v = 0; v < PER; ++v) ps[v] = __builtin_fmaf(x[v], inv, ps[v]);
        if (m > NEG_INF && l == 0) ++used;
        float w = chosen >= 0 ? __builtin_amdgcn_exp2f((value - m) * ROUTE_LOG2E) : 0.0f;
        // NaN among the logits makes the weights NaN
        if (p.normalize) {
            const float all = lanes_sum<LANES>(w);
            w = s == s ? (chosen >= 0 ? w * __builtin_amdgcn_rcpf(all) : 0.0f) : chosen >= 0 ? s : 0.0f;
        } else {
            w *= chosen >= 0 ? inv : 0.0f;
        }
        if (r < rows && l < k) {
            p.index[row * k + l] = chosen;
            p.weight[row * k + l] = w;
            if constexpr (ALL) kept[r * k + l] = chosen;
            if (chosen >= 0) atomicAdd(&counts[chosen], 1);
        }
    }
    __syncthreads();
    // probabilities: rows side by side, then the waves, are added up in order
#pragma unroll
    for (int v = 0; v < PER; ++v) {
        if constexpr (LANES <= 16) ps[v] += __shfl_xor(ps[v], 16);
        if constexpr (LANES <= 32) ps[v] += __shfl_xor(ps[v], 32);
        if (slot == 0) psum[wave * WIDTH + S::expert(l, v)] = ps[v];
    }
    for (int h = LANES; h < 64; h *= 2) used += __shfl_xor(used, h);   // lane 0 of every row counts
    if (lane == 0) used_rows[wave] = used;
    __syncthreads();
    int all_used = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) all_used += used_rows[w];
    for (int e = threadIdx.x; e < E; e += THREADS) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) t += psum[i * WIDTH + e];
        if constexpr (ALL) {
            ptotal[e] = t;
            starts[e] = counts[e];
        } else {
            p.psum[(int64_t)blockIdx.x * E + e] = t;
            p.hist[(int64_t)blockIdx.x * (E + 1) + e] = counts[e];
        }
    }
    if constexpr (!ALL) {
        if (threadIdx.x == 0) p.hist[(int64_t)blockIdx.x * (E + 1) + E] = all_used;
    } else {
        __syncthreads();
        scan_experts(starts, E);
        finish_totals(p, starts, all_used, ptotal);
        Choices<true> mine;
        mine.init(p, kept, rows, SLOTS * WIDTH);
        place_choices(p, row0, mine, starts, starts[E], shared);
    }
}

// The rest for several workgroups: each sums the counts of all and of those before it (every thread
// those of one expert over a run of workgroups; no launch between) and places its choices; one more
// writes the totals.
constexpr int PLACE_THREADS = 1024, PLACE_COUNTERS = 8192;
__global__ __launch_bounds__(PLACE_THREADS) void place_blocks(RouteParams p) {
    static_assert(PLACE_COUNTERS >= 2 * (PLACE_THREADS + ROUTE_MAX_EXPERTS + 1), "runs of counters");
    __shared__ int hist[PLACE_COUNTERS];             // the runs' sums, then the waves' counters
    __shared__ int starts[ROUTE_MAX_EXPERTS + 1], before[ROUTE_MAX_EXPERTS + 1];
    const int E = p.experts, cols = E + 1, me = blockIdx.x;
    const bool totals = me == p.blocks;
    const int row0 = me * p.block_rows;
    Choices<false> mine;
    mine.init(p, p.index + (int64_t)row0 * p.k, totals ? 0 : min(p.block_rows, p.rows - row0), PLACE_COUNTERS);
    const int runs = max(PLACE_THREADS / cols, 1), per = (p.blocks + runs - 1) / runs;
    for (int i = threadIdx.x; i < runs * cols; i += PLACE_THREADS) {   // (one turn, or two with 1024 experts)
        const int run = i / cols, e = i - run * cols;
        const int b0 = min(run * per, p.blocks), b1 = min(b0 + per, p.blocks), bm = min(max(me, b0), b1);
        const int *h = p.hist + e;
        int low = 0, high = 0;
#pragma unroll 16
        for (int b = b0; b < bm; ++b) low += h[(int64_t)b * cols];
#pragma unroll 16
        for (int b = bm; b < b1; ++b) high += h[(int64_t)b * cols];
        hist[2 * i] = low;
        hist[2 * i + 1] = low + high;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < cols; e += PLACE_THREADS) {
        int low = 0, all = 0;
        for (int r = 0; r < runs; ++r) {
            low += hist[2 * (r * cols + e)];
            all += hist[2 * (r * cols + e) + 1];
        }
        before[e] = low;
        starts[e] = all;
    }
    __syncthreads();
    const int used = starts[E];
    __syncthreads();
    scan_experts(starts, E);
    if (totals) {
        float *const ptotal = reinterpret_cast<float *>(before);
        double *const part = reinterpret_cast<double *>(hist);
        static_assert(PLACE_COUNTERS >= 2 * (PLACE_THREADS + ROUTE_MAX_EXPERTS), "runs of sums");
        const int sums = max(PLACE_THREADS / E, 1), each = (p.blocks + sums - 1) / sums;
        for (int i = threadIdx.x; p.loss && i < sums * E; i += PLACE_THREADS) {
            const int run = i / E, e = i - run * E;
            const int b0 = min(run * each, p.blocks), b1 = min(b0 + each, p.blocks);
            double t = 0.0;
#pragma unroll 16
            for (int b = b0; b < b1; ++b) t += p.psum[(int64_t)b * E + e];
            part[i] = t;
        }
        __syncthreads();
        for (int e = threadIdx.x; p.loss && e < E; e += PLACE_THREADS) {
            double t = 0.0;
            for (int r = 0; r < sums; ++r) t += part[r * E + e];
            ptotal[e] = (float)t;
        }
        __syncthreads();
        finish_totals(p, starts, used, ptotal);
        return;
    }
    const int total = starts[E];
    for (int e = threadIdx.x; e < E; e += PLACE_THREADS) before[e] += starts[e];
    __syncthreads();
    place_choices(p, row0, mine, before, total, hist);
}

// d logit_j = p_j (dloss slope_j - S) + c_j, c_j the chosen's share, by the lane of the choice: with
// normalize c = w (dweight - sum w dweight) and S = dloss sum p slope, else c = p dweight and S has their sum
// too.  LDS takes the exponentials to the lanes of the choices, and the shares to those of the experts.
template <class T, int LANES, int PER>
__global__ __launch_bounds__(ROUTE_THREADS) void grad(RouteParams p) {
    constexpr int ROWS = 64 / LANES, SLOTS = ROUTE_WAVES * ROWS, WIDTH = LANES * PER;
    __shared__ __attribute__((aligned(16))) float powers[SLOTS][WIDTH], shares[SLOTS][WIDTH];
    const int E = p.experts, k = p.k;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    using S = Share<T, LANES, PER>;
    const int slot = wave * ROWS + lane / LANES, l = lane % LANES;
    float *const power = powers[slot], *const share = shares[slot];
    float slope[PER];
    const float dloss = p.dloss && p.slope ? p.dloss[0] : 0.0f;
#pragma unroll
    for (int v = 0; v < PER; ++v) {
        const int e = S::expert(l, v);
        slope[v] = p.dloss && p.slope && e < E ? dloss * p.slope[e] : 0.0f;
        share[e] = 0.0f;
    }
    const int step = gridDim.x * SLOTS;
    // a row's loads, side by side; the next row's are under way while one is worked on
    float next[PER], next_dw = 0.0f;
    int next_on = 0, next_at = -1;
    auto fetch = [&](int64_t row) {
        next_on = row < p.rows;
        if (row < p.rows) {
            if (p.mask) next_on = p.mask[row];
            S::load(static_cast<const T *>(p.logits) + row * p.ldl, l, E, next);
            if (p.dweight && l < k) {
                next_at = p.index[row * k + l];
                next_dw = p.dweight[row * k + l];
            }
        }
    };
    // (one wave's lanes exchange their values: its LDS operations execute in order)
    auto order = [&]() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    const int64_t row0 = (int64_t)blockIdx.x * SLOTS + slot;
    fetch(row0);
#pragma unroll 1
    for (int64_t row = row0; row - lane / LANES < p.rows; row += step) {
        const bool on = next_on != 0;
        float x[PER];
#pragma unroll
        for (int v = 0; v < PER; ++v) x[v] = on ? next[v] : NEG_INF;
        const int at = on && next_at >= 0 && next_at < E ? next_at : -1;
        const float dw = next_dw;
        fetch(row + step);
        const float m = lanes_max<LANES>(largest(x));
        const float s = exponentials<LANES>(x, m), inv = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
        float sp = 0.0f;
#pragma unroll
        for (int v = 0; v < PER; ++v) {
            x[v] *= inv;
            power[S::expert(l, v)] = x[v];
            sp = __builtin_fmaf(x[v], slope[v], sp);
        }
        sp = lanes_sum<LANES>(sp);
        order();
        const float mine = at >= 0 ? power[at] : 0.0f;
        float c;
        if (p.normalize) {
            const float all = lanes_sum<LANES>(mine), w = all == 0.0f ? 0.0f : mine * __builtin_amdgcn_rcpf(all);
            const float given = at >= 0 ? dw : 0.0f;
            c = w * (given - lanes_sum<LANES>(w * given));
        } else {
            c = at >= 0 ? mine * dw : 0.0f;
            sp += lanes_sum<LANES>(c);
        }
        if (at >= 0) share[at] = c;
        order();
        float d[PER];
#pragma unroll
        for (int v = 0; v < PER; ++v) d[v] = __builtin_fmaf(x[v], slope[v] - sp, share[S::expert(l, v)]);
        order();
        if (at >= 0) share[at] = 0.0f;               // for the next row
        if (row < p.rows) {
            if (!on) {                               // left out: 0, whatever dloss is
#pragma unroll
                for (int v = 0; v < PER; ++v) d[v] = 0.0f;
            }
            S::store(static_cast<T *>(p.dlogits) + row * p.ldl, l, E, d);
        }
    }
}

template <class T, int LANES, int PER>
hipError_t launch_choose(const RouteParams &p, hipStream_t s) {
    constexpr int THREADS = route_waves(LANES * PER) * 64;
    if (p.blocks == 1) hipLaunchKernelGGL((choose<T, LANES, PER, true>), dim3(1), dim3(THREADS), 0, s, p);
    else hipLaunchKernelGGL((choose<T, LANES, PER, false>), dim3(p.blocks), dim3(THREADS), 0, s, p);
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
    hipLaunchKernelGGL(place_blocks, dim3(p.blocks + 1), dim3(PLACE_THREADS), 0, stream, p);
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
