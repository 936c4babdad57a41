// Drives the plan and run logic of a layer's products, layer norm and routing (host side, sanitizers on)
// over random and edge-case descriptions, with the kernels replaced by layer_stubs.cpp.  Enum fields
// also get out-of-range bits, as a C caller can store them.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>

#include "../../include/gemm.h"

namespace tge {
extern int layer_launches, norm_launches, route_launches;
}

static std::mt19937_64 rng(11);
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
static int64_t ld(int64_t least) { return rng() % 30 && least < INT64_MAX - 2 ? least + (int64_t)(rng() % 3) : size(); }
static void *ptr() { return rng() % 20 ? (void *)(uintptr_t)(4096 * (1 + rng() % 3) + (rng() % 20 ? 0 : rng() % 4)) : nullptr; }
static float *fptr() { return (float *)ptr(); }
static int32_t *iptr() { return (int32_t *)ptr(); }

int main() {
    int failures = 0, made = 0;
    char buf[16];
    char big[256];
    const float nan = std::nanf("");
    for (int i = 0; i < 60000; ++i) {
        const float alpha = rng() % 10 ? 1.0f : nan, beta = rng() % 10 ? (float)pick({0, 0, 1}) : nan;
        gemm_status_t st;
        size_t need = 0;
        if (i % 3 == 0) {
            gemm_layer_desc_t d = {};
            d.rows = size(); d.N = size(); d.K = size(); d.groups = pick({-1, 0, 1, 1, 2, 64, 1000, (int64_t)1 << 20, INT64_MAX});
            const int op = (int)pick({0, 0, 1, 1, 2, -7});
            put(d.op_b, op);
            d.lda = ld(d.K); d.ldb = ld(op ? d.K : d.N); d.ldc = ld(d.N);
            d.stride_b = size(); d.stride_bias = size();
            const int ab = type();
            put(d.ab_type, ab); put(d.cd_type, rng() % 3 ? ab : type());
            put(d.act, (int)pick({0, 1, 2, 3, 4, 5, -1})); put(d.algo, (int)pick({0, 0, 0, 1, 2, 3, 4, 5, 99}));
            d.tile = (int)pick({0, 0, 0, 0, 16, 32, 64, 128, 256});
            gemm_layer_plan_t p = (gemm_layer_plan_t)1;
            const bool whole = rng() % 50;
            st = gemm_layer_plan_create(whole ? &p : nullptr, rng() % 50 ? &d : nullptr);
            if (!whole) continue;
            if ((st == GEMM_STATUS_SUCCESS) != (p != nullptr)) ++failures;
            if (!p) continue;
            if (gemm_layer_plan_describe(p, buf, sizeof buf) || gemm_layer_plan_describe(p, big, sizeof big)) ++failures;
            for (int r = 0; r < 4; ++r) {
                gemm_layer_run(p, ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), iptr(), alpha, beta, nullptr);
                gemm_layer_grad_run(p, ptr(), ptr(), ptr(), ptr(), iptr(), alpha, nullptr);
            }
            gemm_layer_plan_destroy(p);
        } else if (i % 3 == 1) {
            gemm_norm_desc_t d = {};
            d.rows = size(); d.N = size(); d.ldx = ld(d.N); d.ldy = ld(d.N);
            put(d.type, type());
            d.eps = rng() % 10 ? 1e-5f : (float)pick({0, -1}) + (rng() % 2 ? nan : INFINITY);
            gemm_norm_plan_t p = (gemm_norm_plan_t)1;
            st = gemm_norm_plan_create(&p, rng() % 50 ? &d : nullptr);
            if ((st == GEMM_STATUS_SUCCESS) != (p != nullptr)) ++failures;
            if (!p) continue;
            if (gemm_norm_plan_describe(p, buf, sizeof buf) || gemm_norm_workspace_bytes(p, &need)) ++failures;
            for (int r = 0; r < 4; ++r) {
                gemm_norm_run(p, ptr(), fptr(), fptr(), ptr(), fptr(), fptr(), nullptr);
                gemm_norm_grad_run(p, ptr(), ptr(), fptr(), fptr(), fptr(), ptr(), ptr(), fptr(), fptr(), beta, ptr(),
                                   need - (rng() % 9 == 0 && need), nullptr);
            }
            gemm_norm_plan_destroy(p);
        } else {
            gemm_route_desc_t d = {};
            d.rows = size(); d.experts = pick({-1, 0, 1, 3, 8, 16, 17, 64, 100, 128, 256, 512, 1024, 1025, INT64_MAX});
            d.k = pick({-1, 0, 1, 1, 2, 2, 8, 16, 17, INT64_MAX}); d.ldl = ld(d.experts);
            put(d.type, type());
            d.normalize = (int)pick({0, 0, 1, 1, 2});
            gemm_route_plan_t p = (gemm_route_plan_t)1;
            st = gemm_route_plan_create(&p, rng() % 50 ? &d : nullptr);
            if ((st == GEMM_STATUS_SUCCESS) != (p != nullptr)) ++failures;
            if (!p) continue;
            if (gemm_route_plan_describe(p, buf, sizeof buf) || gemm_route_workspace_bytes(p, &need)) ++failures;
            for (int r = 0; r < 4; ++r) {
                gemm_route_run(p, ptr(), (uint8_t *)ptr(), iptr(), fptr(), iptr(), iptr(), iptr(), fptr(), fptr(), ptr(),
                               need - (rng() % 9 == 0 && need), nullptr);
                gemm_route_grad_run(p, ptr(), (uint8_t *)ptr(), iptr(), fptr(), fptr(), fptr(), ptr(), nullptr);
            }
            gemm_route_plan_destroy(p);
        }
        ++made;
    }
    if (made < 1000 || tge::layer_launches < 1000 || tge::norm_launches < 1000 || tge::route_launches < 1000) ++failures;
    std::printf("%d plans, %d + %d + %d launches, %d failures\n", made, tge::layer_launches, tge::norm_launches, tge::route_launches,
                failures);
    return failures != 0;
}
