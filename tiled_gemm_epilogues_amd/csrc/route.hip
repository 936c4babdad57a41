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
// infinity are never chosen, and a row of nothing else is left out.  Bound: the instructions of the
// choice for many rows, launches for few:
// 65536 rows of 128 fp32 logits (34 MB), 8 chosen, 18.6 us, of which the first loads 3, the choice 9 and the
// launch and its end 4, and 10.4 us for the places; one row 5.7 us; the gradient 15.4 us (67 MB and the choices: 4.6 TB/s).
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

// Reduction over a row's lanes, the result in each of them.
template <int LANES, class Op>
__device__ __forceinline__ int over_lanes(int v, Op op) {
    lane_steps<LANES>([&](auto move) { v = op(v, moved<move.value>(v)); });
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
// many waves take part as there are rows of counters for, and choices.  index: the workgroup's choices, in memory
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
        const int chunks = (n + 63) / 64;
        waves = max(min(min((int)blockDim.x / 64, counters / p.experts), chunks), 1);
        const int per = (chunks + waves - 1) / waves;
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
        constexpr int SIDE = 8;                          // (read side by side, then written)
        for (int w = 0; w < waves; w += SIDE) {
            int h[SIDE];
#pragma unroll
            for (int n = 0; n < SIDE; ++n) h[n] = hist[min(w + n, waves - 1) * E + e];
#pragma unroll
            for (int n = 0; n < SIDE; ++n) {
                if (w + n < waves) hist[(w + n) * E + e] = at;
                at += h[n];
            }
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

// Offsets, slope and loss from the totals: starts[E + 1] and the probabilities' sums (LDS), the used
// rows.
__device__ void finish_totals(const RouteParams &p, const int *starts, int used, const float *ptotal) {
    const int E = p.experts;
    for (int e = threadIdx.x; e <= E; e += blockDim.x) p.offsets[e] = starts[e];
    // (in 64 bits: rows have more digits than fp32)
    const double scale = used > 0 ? (double)E / ((double)p.k * used * used) : 0.0;
    if (p.slope)
        for (int e = threadIdx.x; e < E; e += blockDim.x) p.slope[e] = (float)(scale * (starts[e + 1] - starts[e]));
    if (p.loss && threadIdx.x < 64) {
        float s = 0.0f;
        for (int e = threadIdx.x; e < E; e += 64) s = __builtin_fmaf((float)(scale * (starts[e + 1] - starts[e])), ptotal[e], s);
        s = wave_sum(s);
        if (threadIdx.x == 0) p.loss[0] = s;
    }
}

// One step of a row's choice: of the sorted keys of two lanes the LEN largest, sorted, in both.  The
// larger of the one's i-th and the other's last-but-i-th are the largest; they rise and fall once, and
// halving exchanges sort them.  sent: what the other lane takes.
template <int MOVE, int LEN>
__device__ __forceinline__ void merge_lanes(uint32_t (&v)[LEN], const uint32_t (&sent)[LEN]) {
    uint32_t other[LEN];
#pragma unroll
    for (int i = 0; i < LEN; ++i) other[i] = (uint32_t)moved<MOVE>((int)sent[LEN - 1 - i]);
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

// Choice of the j-th largest logits, j < k, of the rows of a wave, AT of them per LANES lanes; on return lane j of
// the u-th of AT parts of the lanes holds the j-th expert of row u (-1: none is left).  A lane's logits
// become keys of 32 bits, their rank with its last bits replaced by the expert, lowest last, so that one
// unsigned comparison orders values and experts and no two keys are equal; each lane sorts its own, then lanes
// merge theirs in pairs (some 35 instructions a step, where taking one maximum after another costs as many
// for each choice: 65536 rows of 128, 8 chosen, 23 us so).  After a merge both lanes have the same keys; so
// with two rows at a time the first merge gives one half of the lanes to each, and the others, and all
// that follows, serve both rows at once.
//
// 16-bit logits lose nothing in the key.  fp32 logits lose their last bits: where two keys in order have the
// same bits left (the first not chosen included) it may be wrong or a tie, and the wave chooses again from
// the logits themselves.  For random logits that is about one row in a thousand.
template <class T, int LANES, int PER, int LEN, int AT>
__device__ __forceinline__ int choose_experts(const float (&x)[AT][PER], int l, int k) {
    using S = Share<T, LANES, PER>;
    constexpr bool EXACT = sizeof(T) == 2;
    constexpr uint32_t LAST = LANES * PER - 1;
    constexpr int PART = LANES / AT;
    static_assert(PART >= LEN, "a lane per choice");
    const bool second = l >= PART;
    const int j = l % PART;
    uint32_t key[AT][PER], all[AT][LEN], v[LEN];
#pragma unroll
    for (int u = 0; u < AT; ++u) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[u][i] = (rank_of(x[u][i]) & ~LAST) | (LAST - S::expert(l, i));
        sort_keys(key[u]);
#pragma unroll
        for (int i = 0; i < LEN; ++i) all[u][i] = i < PER ? key[u][i < PER ? i : 0] : 0u;
    }
    if constexpr (AT == 2) {
        uint32_t sent[LEN];
#pragma unroll
        for (int i = 0; i < LEN; ++i) {
            v[i] = second ? all[1][i] : all[0][i];
            sent[i] = second ? all[0][i] : all[1][i];
        }
        merge_lanes<PART == 8 ? RING + 8 : PART>(v, sent);
    } else {
#pragma unroll
        for (int i = 0; i < LEN; ++i) v[i] = all[0][i];
    }
    lane_steps<PART>([&](auto move) {
        uint32_t sent[LEN];
#pragma unroll
        for (int i = 0; i < LEN; ++i) sent[i] = v[i];
        merge_lanes<move.value>(v, sent);
    });
    uint32_t taken = 0;
#pragma unroll
    for (int i = 0; i < LEN; ++i) taken = j == i ? v[i] : taken;
    if (j >= k) taken = 0;
    int chosen = taken >= LOWEST ? (int)(LAST - (taken & LAST)) : -1;
    if constexpr (!EXACT) {
        // two neighbours of the order with the same bits left
        const uint32_t next = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)taken, 0x101, 0xf, 0xf, true);   // lane j + 1's
        const bool bad = j + 1 < k && next >= LOWEST && (next ^ taken) <= LAST;
        // or more keys with the last one's bits, or above, than were chosen.  No row has fewer, so the
        // numbers over the wave are equal only if they are in every row
        uint32_t kth = v[0];
#pragma unroll
        for (int i = 1; i < LEN; ++i) kth = i < k ? v[i] : kth;
        const uint32_t from = max(kth & ~LAST, LOWEST);
        int above = 0;
        if constexpr (AT == 2) {
            const uint32_t other = (uint32_t)moved<PART == 8 ? RING + 8 : PART>((int)from);
            const uint32_t first = second ? other : from, last = second ? from : other;
#pragma unroll
            for (int i = 0; i < PER; ++i) above += __popcll(__ballot(key[0][i] >= first)) + __popcll(__ballot(key[1][i] >= last));
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) above += __popcll(__ballot(key[0][i] >= from));
        }
        if (__ballot(bad) != 0 || above != __popcll(__ballot(taken >= LOWEST))) {
#pragma unroll 1
            for (int u = 0; u < AT; ++u) {
                float left[PER];
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const float x0 = x[0][i], x1 = x[AT - 1][i], xi = u == 0 ? x0 : x1;
                    left[i] = xi == xi ? xi : NEG_INF;
                }
#pragma unroll 1
                for (int n = 0; n < k; ++n) {
                    const float best = lanes_max<LANES>(largest(left));
                    int at = 1 << 30;
#pragma unroll
                    for (int i = PER - 1; i >= 0; --i) at = left[i] == best ? S::expert(l, i) : at;
                    at = lanes_min<LANES>(at);
                    if (best == NEG_INF) at = -1;
#pragma unroll
                    for (int i = 0; i < PER; ++i) left[i] = S::expert(l, i) == at ? NEG_INF : left[i];
                    chosen = l == u * PART + n ? at : chosen;
                }
            }
        }
    }
    return chosen;
}

// ALL: one workgroup does the whole routing.  A wave works on AT rows per LANES lanes at a time; LEN: the
// most choices.
template <class T, int LANES, int PER, int LEN, int AT, bool ALL>
__global__ __launch_bounds__(route_waves(LANES *PER) * 64) void choose(RouteParams p) {
    constexpr int ROWS = 64 / LANES;                 // groups of lanes
    constexpr int WIDTH = LANES * PER;               // experts, rounded up
    constexpr int WAVES = route_waves(WIDTH), THREADS = WAVES * 64, SLOTS = WAVES * ROWS;
    constexpr int PART = LANES / AT;
    __shared__ int counts[WIDTH];
    __shared__ int starts[WIDTH + 1];
    __shared__ float ptotal[WIDTH];
    // the rows at work, then the waves' summed probabilities, then their counters
    __shared__ __attribute__((aligned(16))) int shared[AT * SLOTS * WIDTH];
    __shared__ int used_rows[WAVES];
    __shared__ int kept[ALL ? route_one_rows(WAVES, LANES) * ROUTE_MAX_K : 1];   // the choices, for their places
    const int E = p.experts, k = p.k;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    using S = Share<T, LANES, PER>;
    const int slot = lane / LANES, l = lane % LANES;
    const int part = l / PART, j = l % PART;         // the row whose j-th choice is this lane's
    const int row0 = blockIdx.x * p.block_rows, rows = min(p.block_rows, p.rows - row0);
    const T *logits = static_cast<const T *>(p.logits) + (int64_t)row0 * p.ldl;
    float *const psum = reinterpret_cast<float *>(shared), *const values = psum + (wave * ROWS + slot) * AT * WIDTH;
    for (int e = threadIdx.x; e < WIDTH; e += THREADS) counts[e] = 0;
    __syncthreads();
    float ps[PER], next[AT][PER];
#pragma unroll
    for (int v = 0; v < PER; ++v) ps[v] = 0.0f;
    int used = 0;
    int next_on[AT];
    // (loads side by side, none waiting for another)
    auto fetch = [&](int r) {
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            const int at = r + u * SLOTS;
            next_on[u] = at < rows;
            if (at < rows) {
                if (p.mask) next_on[u] = p.mask[row0 + at];
                S::load(logits + (int64_t)at * p.ldl, l, E, next[u]);
            }
        }
    };
    const int end = (rows + ROWS - 1) / ROWS * ROWS; // (a wave's rows stay together)
    fetch(wave * ROWS + slot);
#pragma unroll 1
    for (int r = wave * ROWS + slot; r < end; r += AT * SLOTS) {
        float x[AT][PER];
#pragma unroll
        for (int u = 0; u < AT; ++u)
#pragma unroll
            for (int v = 0; v < PER; ++v) x[u][v] = next_on[u] ? next[u][v] : NEG_INF;
        if (end - r > AT * SLOTS) fetch(r + AT * SLOTS);
        // the rows in LDS, where their lanes find the chosen logits
#pragma unroll
        for (int u = 0; u < AT; ++u)
#pragma unroll
            for (int v = 0; v < PER; ++v) values[u * WIDTH + S::expert(l, v)] = x[u][v];
        const int chosen = choose_experts<T, LANES, PER, LEN, AT>(x, l, k);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float value = chosen >= 0 ? values[part * WIDTH + chosen] : 0.0f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        float m = 0.0f, s = 0.0f, inv = 0.0f;
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            const float mu = lanes_max<LANES>(largest(x[u]));
            const float su = exponentials<LANES>(x[u], mu), iu = su == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(su);
            if (mu > NEG_INF) {                      // (a row left out may hold NaN)
#pragma unroll
                for (int v = 0; v < PER; ++v) ps[v] = __builtin_fmaf(x[u][v], iu, ps[v]);
                if (l == 0) ++used;
            }
            m = part == u ? mu : m;
            s = part == u ? su : s;
            inv = part == u ? iu : inv;
        }
        float w = chosen >= 0 ? __builtin_amdgcn_exp2f((value - m) * ROUTE_LOG2E) : 0.0f;
        // NaN among the logits makes the weights NaN
        if (p.normalize) {
            const float all = lanes_sum<PART>(w);
            w = s == s ? (chosen >= 0 ? w * __builtin_amdgcn_rcpf(all) : 0.0f) : chosen >= 0 ? s : 0.0f;
        } else {
            w *= chosen >= 0 ? inv : 0.0f;
        }
        const int at = r + part * SLOTS;
        if (at < rows && j < k) {
            const int64_t to = (int64_t)(row0 + at) * k + j;
            p.index[to] = chosen;
            p.weight[to] = w;
            if constexpr (ALL) kept[at * k + j] = chosen;
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
            p.psum[e * p.stride + blockIdx.x] = t;
            p.hist[e * p.stride + blockIdx.x] = counts[e];
        }
    }
    if constexpr (!ALL) {
        if (threadIdx.x == 0) p.hist[E * p.stride + blockIdx.x] = all_used;
    } else {
        __syncthreads();
        scan_experts(starts, E);
        finish_totals(p, starts, all_used, ptotal);
        Choices<true> mine;
        mine.init(p, kept, rows, SLOTS * WIDTH);
        place_choices(p, row0, mine, starts, starts[E], shared);
    }
}

// The rest for several workgroups: each sums the counts of all and of those before it (no launch between) and
// places its choices; one more writes the totals.  The counts and probabilities of an expert stand side by
// side, p.stride of each: a lane has four, and a wave those of 1 to 64 experts with one load.
constexpr int PLACE_THREADS = 1024, PLACE_COUNTERS = 8192;
template <bool WHOLE>                                // a wave to an expert
__global__ __launch_bounds__(PLACE_THREADS, 8) void place_blocks(RouteParams p) {
    static_assert(ROUTE_MAX_BLOCKS == 64 * 4, "four workgroups to a lane");
    typedef int i32x4a __attribute__((ext_vector_type(4), aligned(4)));
    typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));
    constexpr int WAVES = PLACE_THREADS / 64, SIDE = WHOLE ? 8 : 4;
    __shared__ int hist[PLACE_COUNTERS];             // the waves' counters
    __shared__ int starts[ROUTE_MAX_EXPERTS + 1], before[ROUTE_MAX_EXPERTS + 1];
    const int E = p.experts, me = blockIdx.x;
    const bool totals = me == p.blocks;
    const int row0 = me * p.block_rows;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    float *const ptotal = reinterpret_cast<float *>(before);
    Choices<false> mine;
    mine.init(p, p.index + (int64_t)row0 * p.k, totals ? 0 : min(p.block_rows, p.rows - row0), PLACE_COUNTERS);
    // lanes of an expert (a power of two), experts of a load; this lane's workgroups b0 .. b0 + 3, and how many of
    // them there are, and are before this one
    const int per = WHOLE ? 64 : p.stride / 4, side = 64 / per, sub = WHOLE ? 0 : lane / per, in = lane & (per - 1);
    const int b0 = 4 * in;
    const int have = min(max(p.blocks - b0, 0), 4), low_have = min(max(me - b0, 0), 4);
    const int loads = WHOLE ? E + 1 : (E + side) / side;   // of E + 1 counts
    for (int c = wave; c < loads; c += WAVES * SIDE) {
        i32x4a h[SIDE];
#pragma unroll
        for (int n = 0; n < SIDE; ++n)
            h[n] = *reinterpret_cast<const i32x4a *>(p.hist + min((c + n * WAVES) * side + sub, E) * p.stride + b0);
#pragma unroll
        for (int n = 0; n < SIDE; ++n) {
            if (c + n * WAVES >= loads) break;
            const int e = (c + n * WAVES) * side + sub;
            int all = 0, low = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                all += (WHOLE || e <= E) && i < have ? h[n][i] : 0;
                low += (WHOLE || e <= E) && i < low_have ? h[n][i] : 0;
            }
            // an expert's sum is what the running sum grows by over its lanes
            all = wave_scan_add(all);
            low = wave_scan_add(low);
            if constexpr (!WHOLE) {
                const int all_to = __shfl_up(all, per), low_to = __shfl_up(low, per);
                all -= lane >= per ? all_to : 0;
                low -= lane >= per ? low_to : 0;
            }
            if (in == per - 1 && (WHOLE || e <= E)) {
                starts[e] = all;
                if (!totals) before[e] = low;
            }
        }
    }
    if (totals && p.loss) {
        for (int c = wave; c < loads; c += WAVES * SIDE) {
            f32x4a q[SIDE];
#pragma unroll
            for (int n = 0; n < SIDE; ++n)
                q[n] = *reinterpret_cast<const f32x4a *>(p.psum + min((c + n * WAVES) * side + sub, E - 1) * p.stride + b0);
#pragma unroll
            for (int n = 0; n < SIDE; ++n) {
                if (c + n * WAVES >= loads) break;
                const int e = (c + n * WAVES) * side + sub;
                float t = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) t += i < have ? q[n][i] : 0.0f;
                if constexpr (WHOLE) t = wave_sum(t);
                else
                    for (int s = per / 2; s > 0; s /= 2) t += __shfl_xor(t, s);
                if (in == 0 && e < E) ptotal[e] = t;
            }
        }
    }
    __syncthreads();
    const int used = starts[E];
    __syncthreads();
    scan_experts(starts, E);
    if (totals) {
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
            if (m == NEG_INF) {                      // left out: 0, whatever its logits and dloss are
#pragma unroll
                for (int v = 0; v < PER; ++v) d[v] = 0.0f;
            }
            S::store(static_cast<T *>(p.dlogits) + row * p.ldl, l, E, d);
        }
    }
}

template <class T, int LANES, int PER, int LEN>
hipError_t launch_choose(const RouteParams &p, hipStream_t s) {
    constexpr int WIDTH = LANES * PER, WAVES = route_waves(WIDTH), SLOTS = WAVES * 64 / LANES;
    // two rows at a time where every wave has them (us, one and two: 131072 rows of 16, 2 chosen, 22.0 and 17.2;
    // 65536 of 64, 6 chosen, 20.9 and 18.5; 16384 of 256, 8 chosen, 24.7 and 23.4; but 16384 of 64, one to a wave,
    // 13.1 and 14.7) and the registers for them (16384 of 1024, 16 chosen, 103 and 117)
    constexpr bool PAIRS = LANES / 2 >= LEN && WIDTH <= 512;
    const dim3 grid(p.blocks), threads(WAVES * 64);
    if (p.blocks == 1) {
        hipLaunchKernelGGL((choose<T, LANES, PER, LEN, 1, true>), grid, threads, 0, s, p);
        return hipGetLastError();
    }
    if constexpr (PAIRS) {
        if (p.block_rows >= 2 * SLOTS) {
            hipLaunchKernelGGL((choose<T, LANES, PER, LEN, 2, false>), grid, threads, 0, s, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((choose<T, LANES, PER, LEN, 1, false>), grid, threads, 0, s, p);
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
        else return p.k <= 8 ? launch_choose<T, L, P, 8>(p, stream) : launch_choose<T, L, P, ROUTE_MAX_K>(p, stream)
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
    if (p.stride == ROUTE_MAX_BLOCKS) hipLaunchKernelGGL(place_blocks<true>, dim3(p.blocks + 1), dim3(PLACE_THREADS), 0, stream, p);
    else hipLaunchKernelGGL(place_blocks<false>, dim3(p.blocks + 1), dim3(PLACE_THREADS), 0, stream, p);
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
