"""The C ABI of the grouped and 4-bit products on the CPU: plan creation and its refusals, the runs'
refusals (they return before any launch), kernel choice, grid bounds, and the binding's tensor
checks.  None of these calls reaches the GPU."""
import random
import re

import numpy as np
import pytest
import torch

import tiled_gemm_epilogues_amd as tge

OK, INVALID, UNSUPPORTED = tge.STATUS_SUCCESS, tge.STATUS_INVALID_VALUE, tge.STATUS_NOT_SUPPORTED
BIG = 1 << 31


def rows_plan(**kw):
    a = dict(rows=64, N=64, K=64, groups=4, op_b="N", lda=64, ldb=64, ldc=64, stride_b=4096,
             stride_bias=64, ab_type="f16", cd_type="f16", epilogue="none", algo="auto", tile=0)
    a.update(kw)
    st, h = tge.gemm_grouped_plan_create(**a)
    assert (st == OK) == bool(h)
    return st, h


def grad_plan(**kw):
    a = dict(rows=64, M=64, N=64, groups=4, lda=64, ldb=64, ldc=64, stride_c=4096, ab_type="f16",
             cd_type="f32", algo="auto", tile=0)
    a.update(kw)
    st, h = tge.gemm_grouped_grad_plan_create(**a)
    assert (st == OK) == bool(h)
    return st, h


def quant_plan(**kw):
    a = dict(rows=64, N=64, K=128, block=64, groups=4, lda=128, ldq=64, lds=2, ldc=64, stride_q=4096,
             stride_s=128, stride_bias=64, ab_type="f16", cd_type="f16", epilogue="none", zeros=0,
             algo="auto", tile=0)
    a.update(kw)
    st, h = tge.gemm_quant_plan_create(**a)
    assert (st == OK) == bool(h)
    return st, h


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(N=-1), dict(K=-1), dict(groups=0), dict(groups=-3), dict(lda=63), dict(ldb=63),
    dict(op_b="T", ldb=63), dict(ldc=63), dict(stride_b=-1), dict(stride_bias=-1), dict(op_b=2),
    dict(ab_type=9), dict(cd_type=-1), dict(epilogue=5), dict(epilogue=-1), dict(algo=8), dict(algo="split"),
    dict(algo="nosplit"), dict(algo="kmajor"), dict(tile=128), dict(algo="fast", tile=32),
    dict(algo="staged", tile=256), dict(algo="general", tile=256), dict(algo="skinny", tile=48),
    dict(algo="skinny", tile=16), dict(op_b="T", algo="skinny", tile=32), dict(K=0, lda=0)])
def test_rows_invalid(kw):
    assert rows_plan(**kw)[0] == INVALID


@pytest.mark.parametrize("kw", [
    dict(ab_type="i8", cd_type="i32"), dict(ab_type="f16", cd_type="bf16"), dict(ab_type="f32", cd_type="f16"),
    dict(ab_type="cf16", cd_type="cf32"), dict(rows=BIG), dict(lda=BIG), dict(groups=1 << 20),
    dict(K=1 << 16, lda=1 << 16, ldb=1 << 15, N=1 << 15, ldc=1 << 15), dict(stride_b=1 << 61),
    dict(rows=BIG - 1, N=1 << 20, ldc=1 << 20, ldb=1 << 20)])
def test_rows_not_supported(kw):
    assert rows_plan(**kw)[0] == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(M=-1), dict(N=-1), dict(groups=0), dict(lda=63), dict(ldb=63), dict(ldc=63),
    dict(stride_c=4095), dict(stride_c=-1), dict(ab_type=-1), dict(cd_type=9), dict(algo="skinny"),
    dict(algo="split"), dict(algo=-1), dict(tile=64), dict(algo="fast", tile=32), dict(M=0, lda=0)])
def test_grad_invalid(kw):
    assert grad_plan(**kw)[0] == INVALID


@pytest.mark.parametrize("kw", [dict(ab_type="i8", cd_type="i32"), dict(ab_type="bf16", cd_type="f16"),
                                dict(rows=BIG), dict(ldb=BIG), dict(stride_c=1 << 61), dict(groups=1 << 20)])
def test_grad_not_supported(kw):
    assert grad_plan(**kw)[0] == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(N=-1), dict(K=-64), dict(groups=0), dict(block=0), dict(block=-32), dict(K=96),
    dict(lda=127), dict(ldq=63), dict(lds=1), dict(ldc=63), dict(stride_q=-1), dict(stride_s=-1),
    dict(stride_bias=-1), dict(epilogue="gate"), dict(epilogue=-1), dict(zeros=2), dict(zeros=-1),
    dict(algo="general"), dict(algo="staged"), dict(algo="skinny", tile=32), dict(algo="fast", tile=256),
    dict(tile=16), dict(ab_type=9)])
def test_quant_invalid(kw):
    assert quant_plan(**kw)[0] == INVALID


@pytest.mark.parametrize("kw", [
    dict(ab_type="f32", cd_type="f32"), dict(ab_type="i8", cd_type="i32"), dict(cd_type="bf16"),
    dict(block=16, lds=8), dict(block=96, K=192, lda=192, ldq=96), dict(rows=BIG), dict(ldc=BIG),
    dict(K=1 << 23, lda=1 << 23, ldq=1 << 22, lds=1 << 17), dict(stride_q=1 << 61), dict(groups=1 << 20),
    dict(rows=BIG - 1, N=1 << 20, ldc=1 << 20)])
def test_quant_not_supported(kw):
    assert quant_plan(**kw)[0] == UNSUPPORTED


def test_null_arguments():
    L = tge.lib()
    for fn in (L.gemm_grouped_plan_create, L.gemm_grouped_grad_plan_create, L.gemm_quant_plan_create):
        assert fn(None, None) == INVALID
        import ctypes
        h = ctypes.c_void_p(1)
        assert fn(ctypes.byref(h), None) == INVALID and h.value is None
    assert tge.gemm_grouped_plan_destroy(None) == OK
    assert tge.gemm_quant_plan_destroy(None) == OK
    assert tge.gemm_grouped_plan_describe(None)[0] == INVALID
    assert tge.gemm_quant_plan_describe(None)[0] == INVALID


P, NAN = 4096, float("nan")       # a pointer that no refused call follows


def test_rows_run_refusals():
    _, h = rows_plan(epilogue="bias")
    _, gate = rows_plan(epilogue="gate")
    _, grad = grad_plan()
    run = tge.gemm_grouped_run
    good = dict(plan=h, A=P, B=P, C=None, D=P, bias=P, offsets=P, alpha=1.0, beta=0.0, stream=None)
    for bad in (dict(plan=None), dict(plan=grad), dict(A=None), dict(B=None), dict(D=None), dict(bias=None),
                dict(offsets=None), dict(beta=1.0), dict(alpha=NAN), dict(beta=NAN), dict(A=P + 1),
                dict(B=P + 1), dict(D=P + 1), dict(bias=P + 2), dict(offsets=P + 2),
                dict(beta=1.0, C=P + 1), dict(plan=gate), dict(plan=gate, C=P, beta=1.0)):
        assert run(**{**good, **bad}) == INVALID, bad
    # nothing to write: no pointer is looked at
    for kw in (dict(rows=0), dict(N=0)):
        st, e = rows_plan(**kw)
        assert st == OK
        assert run(e, None, None, None, None, None, None, 1.0, 0.0, None) == OK
        tge.gemm_grouped_plan_destroy(e)
    for x in (h, gate, grad):
        tge.gemm_grouped_plan_destroy(x)


def test_grad_run_refusals():
    _, h = grad_plan()
    _, rows = rows_plan()
    run = tge.gemm_grouped_grad_run
    good = dict(plan=h, A=P, B=P, C=None, D=P, bias_grad=P, offsets=P, alpha=1.0, beta=0.0, stream=None)
    for bad in (dict(plan=None), dict(plan=rows), dict(A=None), dict(B=None), dict(D=None), dict(offsets=None),
                dict(beta=1.0), dict(alpha=NAN), dict(A=P + 1), dict(D=P + 2), dict(bias_grad=P + 2)):
        assert run(**{**good, **bad}) == INVALID, bad
    for x in (h, rows):
        tge.gemm_grouped_plan_destroy(x)


def test_quant_run_refusals():
    _, h = quant_plan(epilogue="bias", zeros=1)
    run = tge.gemm_quant_run
    good = dict(plan=h, A=P, Q=P, scales=P, zeros=P, C=None, D=P, bias=P, offsets=P, alpha=1.0, beta=0.0,
                stream=None)
    for bad in (dict(plan=None), dict(A=None), dict(Q=None), dict(scales=None), dict(zeros=None), dict(D=None),
                dict(bias=None), dict(offsets=None), dict(beta=1.0), dict(alpha=NAN), dict(A=P + 1),
                dict(scales=P + 1), dict(D=P + 1), dict(offsets=P + 1), dict(bias=P + 1)):
        assert run(**{**good, **bad}) == INVALID, bad
    tge.gemm_quant_plan_destroy(h)
    st, e = quant_plan(rows=0)
    assert run(e, None, None, None, None, None, None, None, None, 1.0, 0.0, None) == OK
    tge.gemm_quant_plan_destroy(e)


def test_plain_plans_refuse_the_gate():
    assert tge.gemm_plan_create(64, 64, 64, "N", "N", 64, 64, 64, "f16", "f16", "gate")[0] == INVALID


def _kernel(plan):
    return plan.describe().split(" ")[3]


def test_kernel_choice():
    G, W = tge.GroupedPlan, tge.GroupedGradPlan
    assert _kernel(G(8, 1024, 2048, 16, "T")) == "gemm_rows16_16x16"
    assert _kernel(G(64, 2048, 4096, 64, "T")) == "gemm_rows16_16x64"
    assert _kernel(G(64, 2048, 4096, 64, "N")) == "gemm_rows16_16x64"
    assert _kernel(G(1, 2048, 4096, 1, "N")) == "gemm_rows16_16x32"
    assert _kernel(G(2048, 2048, 4096, 64, "T")) == "gemm_fast_128x128"
    assert _kernel(G(32768, 4096, 4096, 8, "T")) == "gemm_fast_256x256"
    assert _kernel(G(4096, 4096, 4096, 1, "T")) == "gemm_fast_256x256"
    assert _kernel(G(5120, 4096, 4096, 1, "T")) == "gemm_fast_128x128"
    assert _kernel(G(30000, 4095, 4096, 8, "N")) == "gemm_fast_128x128_rs"
    assert _kernel(G(3001, 777, 1001, 7, "N", cd="f32")) == "gemm_fast_64x64_rs"
    assert _kernel(G(1000, 1000, 1000, 4, "N")) == "gemm_fast_64x64"
    assert _kernel(G(3000, 777, 1001, 7, "T", ab="f32", cd="f32")).startswith("gemm_mfma")
    assert _kernel(W(16384, 4096, 2048, 16)) == "gemm_fast_128x128"
    assert _kernel(W(16384, 4095, 2048, 16)) == "gemm_fast_128x128_rs"
    assert _kernel(W(3000, 1001, 777, 7)) == "gemm_fast_64x64_rs"
    assert _kernel(W(40, 1955, 7260, 4)) == "gemm_fast_128x128_rs"
    assert _kernel(W(1003, 1024, 704, 8)) == "gemm_fast_64x64"
    assert _kernel(W(32768, 4096, 4096, 4)) == "gemm_fast_256x256"
    assert _kernel(W(32768, 4096, 4096, 1)) == "gemm_fast_256x256"
    assert _kernel(W(8192, 5120, 4096, 1)) == "gemm_fast_128x128"
    assert _kernel(W(16384, 4, 2048, 16)).startswith("gemm_mfma")
    # a pinned kernel whose preconditions do not hold: the general one
    assert _kernel(G(64, 7, 64, 2, "N", algo="skinny")).startswith("gemm_mfma")
    assert _kernel(G(64, 64, 7, 2, "N", algo="fast")).startswith("gemm_mfma")
    Q = lambda *a, **k: tge.QuantPlan(*a, **k).describe().split(" ")[0]
    assert Q(1, 4096, 4096, 128) == "quant_rows_16x16"
    assert Q(16, 16384, 4096, 64) == "quant_rows_16x64"
    assert Q(2000, 4096, 4096, 128) == "quant_tile_128x128"
    assert Q(635, 120, 5056, 32) == "quant_rows_16x16"


def test_grid_covers_every_split_of_the_rows():
    # the launch is sized from rows and groups alone: no split of the rows may need more tiles
    rng = random.Random(3)
    for _ in range(300):
        E, T, N = rng.randint(1, 90), rng.randint(1, 3000), rng.randint(1, 600)
        algo, tile = rng.choice([("fast", 128), ("fast", 256), ("skinny", 0), ("general", 64), ("auto", 0)])
        p = tge.GroupedPlan(T, N, 64, E, "T", algo=algo, tile=tile)
        bm, bn = map(int, re.search(r"tile (\d+)x(\d+)", p.describe()).groups())
        grid = int(re.search(r"grid (\d+)", p.describe()).group(1))
        for _ in range(20):
            w = np.array([rng.random() ** rng.choice([1, 8]) for _ in range(E)])
            used = rng.choice([T, rng.randint(0, T)])
            counts = np.random.default_rng(rng.randrange(1 << 30)).multinomial(used, w / w.sum())
            if rng.random() < 0.3:      # the worst split: ranges of one row, and one of the rest
                counts = np.zeros(E, int)
                counts[: min(E, T)] = 1
                counts[0] += T - counts.sum()
            assert int(np.ceil(counts / bm).sum()) * -(-N // bn) <= grid


def test_binding_checks():
    p = tge.GroupedPlan(10, 8, 16, 3, "N", ldc=12, cd="f32", epilogue="bias")
    p.check("A", torch.zeros(10, 16, dtype=torch.float16))
    p.check("B", torch.zeros(3, 16, 8, dtype=torch.float16))
    p.check("D", torch.zeros(10, 12))
    p.check("D", torch.zeros(9 * 12 + 8))
    p.check("offsets", torch.zeros(4, dtype=torch.int32))
    for what, t, err in (("A", torch.zeros(10, 16), TypeError), ("A", torch.zeros(9, 16, dtype=torch.float16), ValueError),
                         ("A", torch.zeros(16, 10, dtype=torch.float16).t(), ValueError),
                         ("B", torch.zeros(2, 16, 8, dtype=torch.float16), ValueError),
                         ("D", torch.zeros(10, 8), ValueError), ("bias", torch.zeros(23), ValueError),
                         ("bias", torch.zeros(24, dtype=torch.float16), TypeError),
                         ("offsets", torch.zeros(3, dtype=torch.int32), ValueError),
                         ("offsets", torch.zeros(4, dtype=torch.int64), TypeError)):
        with pytest.raises(err):
            p.check(what, t)
    g = tge.GroupedGradPlan(10, 8, 16, 3)
    g.check("bias_grad", torch.zeros(3, 16))
    for what, t in (("A", torch.zeros(10, 16, dtype=torch.float16)), ("D", torch.zeros(2, 8, 16)),
                    ("bias_grad", torch.zeros(47))):
        with pytest.raises(ValueError):
            g.check(what, t)
    q = tge.QuantPlan(5, 8, 128, 32, 2, zeros=True, ab="bf16", cd="bf16")
    q.check("Q", torch.zeros(2, 8, 64, dtype=torch.uint8))
    q.check("zeros", torch.zeros(2, 8, 4, dtype=torch.uint8))
    for what, t, err in (("Q", torch.zeros(2, 8, 128, dtype=torch.uint8), ValueError),
                         ("Q", torch.zeros(2, 8, 64, dtype=torch.int8), TypeError),
                         ("scales", torch.zeros(2, 8, 4, dtype=torch.float16), TypeError),
                         ("zeros", torch.zeros(1, 8, 4, dtype=torch.uint8), ValueError)):
        with pytest.raises(err):
            q.check(what, t)
    for cls, args in ((tge.GroupedPlan, (10, 8, 16, 0)), (tge.GroupedGradPlan, (10, 8, 16, 0)),
                      (tge.QuantPlan, (10, 8, 16, 0)), (tge.QuantPlan, (10, 8, 100, 32))):
        with pytest.raises(tge.GemmError):
            cls(*args)
