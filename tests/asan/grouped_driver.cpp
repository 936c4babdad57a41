// Drives the plan and run logic of the grouped and 4-bit products (host side, sanitizers on) over
// random and edge-case descriptions, with the kernels replaced by grouped_stubs.cpp.  Enum fields
// also get out-of-range bits, as a C caller can store them.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>

#include "../../include/gemm.h"

namespace tge {
extern int grouped_launches;
}

static std::mt19937_64 rng(7);
static int64_t pick(std::initializer_list<int64_t> v) {
    auto it = v.begin();
    std::advance(it, rng() % v.size());
    return *it;
}
static int64_t size() {
    if (rng() % 40) return pick({0, 1, 7, 8, 31, 32, 64, 65, 128, 1000, 4096, 16384});
    return pick({-1, (int64_t)1 << 23, ((int64_t)1 << 31) - 1, (int64_t)1 << 31, INT64_MAX, INT64_MIN});
}
static int type() { return (int)pick(rng() % 20 ? std::initializer_list<int64_t>{0, 1, 2} : std::initializer_list<int64_t>{3, 9, -1}); }
template <class E>
static void put(E &e, int v) { memcpy(&e, &v, sizeof v); }

int main() {
    int failures = 0, made = 0, runs = 0;
    char buf[16];
    char big[256];
    const auto ld = [](int64_t least) { return rng() % 30 && least < INT64_MAX - 2 ? least + (int64_t)(rng() % 3) : size(); };
    const auto ptr = []() { return rng() % 20 ? (void *)(uintptr_t)(4096 + (rng() % 20 ? 0 : rng() % 4)) : nullptr; };
    for (int i = 0; i < 60000; ++i) {
        const float alpha = rng() % 10 ? 1.0f : 0.0f / 0.0f, beta = (float)pick({0, 0, 1});
        gemm_grouped_plan_t g = (gemm_grouped_plan_t)1;
        gemm_status_t st;
        if (i % 3 == 0) {
            gemm_grouped_desc_t d = {};
            d.rows = size(); d.N = size(); d.K = size(); d.groups = pick({-1, 0, 1, 2, 64, 1000, (int64_t)1 << 20, INT64_MAX});
            const int op = (int)pick({0, 0, 1, 1, 2, -7});
            put(d.op_b, op);
            d.lda = ld(d.K); d.ldb = ld(op ? d.K : d.N); d.ldc = ld(d.N);
            d.stride_b = size(); d.stride_bias = size();
            const int ab = type();
            put(d.ab_type, ab); put(d.cd_type, rng() % 3 ? ab : type());
            put(d.epilogue, (int)pick({0, 1, 2, 3, 4, 5, -1})); put(d.algo, (int)pick({0, 0, 0, 1, 2, 3, 4, 5, 99}));
            d.tile = (int)pick({0, 0, 0, 0, 16, 32, 64, 128, 256});
            st = gemm_grouped_plan_create(rng() % 50 ? &g : nullptr, rng() % 50 ? &d : nullptr);
        } else if (i % 3 == 1) {
            gemm_grouped_grad_desc_t d = {};
            d.rows = size(); d.M = size(); d.N = size(); d.groups = pick({-1, 0, 1, 2, 64, 1000, (int64_t)1 << 20});
            d.lda = ld(d.M); d.ldb = ld(d.N); d.ldc = ld(d.N);
            d.stride_c = rng() % 3 && d.M > 0 && d.M < 1 << 20 && d.ldc > 0 && d.ldc < 1 << 20 ? d.M * d.ldc : size();
            const int ab = type();
            put(d.ab_type, ab); put(d.cd_type, rng() % 3 ? ab : type());
            put(d.algo, (int)pick({0, 0, 0, 1, 2, 3, 4, 99})); d.tile = (int)pick({0, 0, 64, 128, 256});
            st = gemm_grouped_grad_plan_create(&g, &d);
        } else {
            gemm_quant_desc_t d = {};
            d.rows = size(); d.N = size(); d.block = pick({-1, 0, 16, 32, 32, 64, 64, 128, 128, 256, 96, (int64_t)1 << 22});
            d.K = d.block > 0 && rng() % 4 ? d.block * (int64_t)(rng() % 40) : size();
            d.groups = pick({-1, 0, 1, 1, 2, 64, (int64_t)1 << 20});
            d.lda = ld(d.K); d.ldq = ld(d.K / 2); d.lds = ld(d.block > 0 ? d.K / d.block : 0); d.ldc = ld(d.N);
            d.stride_q = size(); d.stride_s = size(); d.stride_bias = size();
            const int ab = type();
            put(d.ab_type, ab); put(d.cd_type, rng() % 3 ? ab : type());
            put(d.epilogue, (int)pick({0, 1, 2, 3, 4, -1})); d.zeros = (int)pick({0, 1, 2});
            put(d.algo, (int)pick({0, 0, 0, 1, 4, 3, 99})); d.tile = (int)pick({0, 0, 16, 64, 128});
            gemm_quant_plan_t q = (gemm_quant_plan_t)1;
            st = gemm_quant_plan_create(&q, &d);
            if ((st == GEMM_STATUS_SUCCESS) != (q != nullptr)) ++failures;
            if (st == GEMM_STATUS_SUCCESS) {
                ++made;
                if (gemm_quant_plan_describe(q, buf, sizeof buf) || gemm_quant_plan_describe(q, big, sizeof big)) ++failures;
                for (int r = 0; r < 4; ++r) {
                    gemm_quant_run(q, ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), (const int32_t *)ptr(), alpha, beta, nullptr);
                    ++runs;
                }
            }
            gemm_quant_plan_destroy(q);
            continue;
        }
        if (g != (gemm_grouped_plan_t)1 && (st == GEMM_STATUS_SUCCESS) != (g != nullptr)) ++failures;
        if (st != GEMM_STATUS_SUCCESS) continue;
        ++made;
        if (gemm_grouped_plan_describe(g, buf, sizeof buf) || gemm_grouped_plan_describe(g, big, sizeof big)) ++failures;
        for (int r = 0; r < 4; ++r) {
            gemm_grouped_run(g, ptr(), ptr(), ptr(), ptr(), ptr(), (const int32_t *)ptr(), alpha, beta, nullptr);
            gemm_grouped_grad_run(g, ptr(), ptr(), ptr(), ptr(), (float *)ptr(), (const int32_t *)ptr(), alpha, beta, nullptr);
            ++runs;
        }
        gemm_grouped_plan_destroy(g);
    }
    if (made < 1000 || tge::grouped_launches < 1000) ++failures;
    std::printf("%d plans, %d runs, %d launches, %d failures\n", made, runs, tge::grouped_launches, failures);
    return failures != 0;
}
