"""The C ABI of a layer's products, layer norm and routing on the CPU: plan creation and its refusals, the
runs' refusals (they return before any launch), kernel choice, grid bounds, workspace sizes, and the
binding's tensor checks.  None of these calls reaches the GPU."""
import ctypes
import random
import re

import numpy as np
import pytest
import torch

import tiled_gemm_epilogues_amd as tge

OK, INVALID, UNSUPPORTED = tge.STATUS_SUCCESS, tge.STATUS_INVALID_VALUE, tge.STATUS_NOT_SUPPORTED
BIG = 1 << 31
HUGE = (1 << 63) - 1
P, NAN, INF = 4096, float("nan"), float("inf")       # a pointer that no refused call follows


def layer_plan(**kw):
    a = dict(rows=64, N=64, K=64, groups=4, op_b="N", lda=64, ldb=64, ldc=64, stride_b=4096,
             stride_bias=64, ab_type="f16", cd_type="f16", act="gelu", algo="auto", tile=0)
    a.update(kw)
    st, h = tge.gemm_layer_plan_create(**a)
    assert (st == OK) == bool(h)
    return st, h


def norm_plan(**kw):
    a = dict(rows=64, N=64, ldx=64, ldy=64, type="bf16", eps=1e-5)
    a.update(kw)
    st, h = tge.gemm_norm_plan_create(**a)
    assert (st == OK) == bool(h)
    return st, h


def route_plan(**kw):
    a = dict(rows=64, experts=16, k=2, ldl=16, type="f32", normalize=0)
    a.update(kw)
    st, h = tge.gemm_route_plan_create(**a)
    assert (st == OK) == bool(h)
    return st, h


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(N=-1), dict(K=-1), dict(groups=0), dict(groups=-3), dict(lda=63), dict(ldb=63),
    dict(op_b="T", ldb=63), dict(ldc=63), dict(stride_b=-1), dict(stride_bias=-1), dict(op_b=2), dict(op_b=-1),
    dict(ab_type=9), dict(cd_type=-1), dict(act=5), dict(act=-1), dict(algo=8), dict(algo="split"),
    dict(algo="nosplit"), dict(algo="kmajor"), dict(tile=128), dict(algo="fast", tile=32),
    dict(algo="staged", tile=256), dict(algo="general", tile=256), dict(algo="skinny", tile=48),
    dict(algo="skinny", tile=16), dict(op_b="T", algo="skinny", tile=32), dict(K=0, lda=0),
    dict(rows=-(1 << 63)), dict(N=0, ldc=0)])
def test_layer_invalid(kw):
    assert layer_plan(**kw)[0] == INVALID


@pytest.mark.parametrize("kw", [
    dict(ab_type="i8", cd_type="i32"), dict(ab_type="f16", cd_type="bf16"), dict(ab_type="f32", cd_type="f16"),
    dict(ab_type="cf16", cd_type="cf32"), dict(rows=BIG), dict(rows=HUGE), dict(lda=BIG), dict(ldc=HUGE),
    dict(groups=1 << 20), dict(K=1 << 16, lda=1 << 16, ldb=1 << 15, N=1 << 15, ldc=1 << 15),
    dict(stride_b=1 << 61), dict(stride_bias=1 << 61), dict(rows=BIG - 1, N=1 << 20, ldc=1 << 20, ldb=1 << 20)])
def test_layer_not_supported(kw):
    assert layer_plan(**kw)[0] == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(N=-1), dict(ldx=63), dict(ldy=63), dict(ldx=-1), dict(type=9), dict(type=-1), dict(eps=-1e-9),
    dict(eps=NAN), dict(eps=INF), dict(eps=-INF), dict(N=0, ldx=0), dict(rows=-(1 << 63))])
def test_norm_invalid(kw):
    assert norm_plan(**kw)[0] == INVALID


@pytest.mark.parametrize("kw", [
    dict(type="i8"), dict(type="i32"), dict(type="cf16"), dict(type="df32"), dict(rows=BIG), dict(rows=BIG - (1 << 20)),
    dict(rows=HUGE), dict(N=32769, ldx=32769, ldy=32769), dict(type="f32", N=16385, ldx=16385, ldy=16385),
    dict(N=HUGE, ldx=HUGE, ldy=HUGE), dict(ldx=BIG), dict(ldy=BIG)])
def test_norm_not_supported(kw):
    assert norm_plan(**kw)[0] == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(experts=0), dict(experts=-4), dict(k=0), dict(k=17), dict(ldl=15), dict(type=9), dict(type=-1),
    dict(normalize=2), dict(normalize=-1), dict(rows=-(1 << 63))])
def test_route_invalid(kw):
    assert route_plan(**kw)[0] == INVALID


@pytest.mark.parametrize("kw", [
    dict(type="i8"), dict(type="cf32"), dict(experts=1025, ldl=1025), dict(experts=64, ldl=64, k=17),
    dict(rows=BIG), dict(rows=1 << 30), dict(rows=HUGE), dict(ldl=BIG), dict(rows=BIG - (1 << 20), k=1)])
def test_route_not_supported(kw):
    assert route_plan(**kw)[0] == UNSUPPORTED


def test_null_arguments():
    L = tge.lib()
    for kind in ("layer", "norm", "route"):
        create = getattr(L, f"gemm_{kind}_plan_create")
        assert create(None, None) == INVALID
        h = ctypes.c_void_p(1)
        assert create(ctypes.byref(h), None) == INVALID and h.value is None
        assert getattr(tge, f"gemm_{kind}_plan_destroy")(None) == OK
        assert getattr(tge, f"gemm_{kind}_plan_describe")(None)[0] == INVALID
    _, n = norm_plan()
    _, r = route_plan()
    for kind, h in (("norm", n), ("route", r)):
        assert getattr(tge, f"gemm_{kind}_workspace_bytes")(None)[0] == INVALID
        assert getattr(L, f"gemm_{kind}_workspace_bytes")(h, None) == INVALID
        assert getattr(L, f"gemm_{kind}_plan_describe")(h, None, 4) == INVALID
    tge.gemm_norm_plan_destroy(n)
    tge.gemm_route_plan_destroy(r)


def refused(run, good, bads):
    for bad in bads:
        assert run(**{**good, **bad}) == INVALID, bad


def test_layer_run_refusals():
    _, h = layer_plan()
    good = dict(plan=h, A=P, B=P, C=None, D=P, Z=None, bias=P, offsets=P, alpha=1.0, beta=0.0, stream=None)
    refused(tge.gemm_layer_run, good, (
        dict(plan=None), dict(A=None), dict(B=None), dict(D=None), dict(offsets=None), dict(beta=1.0), dict(alpha=NAN),
        dict(beta=NAN), dict(A=P + 1), dict(B=P + 1), dict(D=P + 1), dict(bias=P + 2), dict(offsets=P + 2),
        dict(beta=1.0, C=P + 1), dict(Z=P + 1), dict(Z=P), dict(Z=2 * P, C=2 * P, beta=1.0)))
    good = dict(plan=h, A=P, B=P, Z=P, D=P, offsets=P, alpha=1.0, stream=None)
    refused(tge.gemm_layer_grad_run, good, (
        dict(plan=None), dict(A=None), dict(B=None), dict(D=None), dict(Z=None), dict(offsets=None), dict(alpha=NAN),
        dict(A=P + 1), dict(B=P + 1), dict(D=P + 1), dict(Z=P + 1), dict(offsets=P + 1)))
    # nothing to write: no pointer is looked at
    for kw in (dict(rows=0), dict(N=0)):
        st, e = layer_plan(**kw)
        assert st == OK
        assert tge.gemm_layer_run(e, None, None, None, None, None, None, None, 1.0, 0.0, None) == OK
        assert tge.gemm_layer_grad_run(e, None, None, None, None, None, 1.0, None) == OK
        tge.gemm_layer_plan_destroy(e)
    tge.gemm_layer_plan_destroy(h)


def test_norm_run_refusals():
    _, h = norm_plan(type="f32")
    good = dict(plan=h, X=P, weight=P, bias=P, Y=P, mean=P, rstd=P, stream=None)
    refused(tge.gemm_norm_run, good, (
        dict(plan=None), dict(X=None), dict(Y=None), dict(X=P + 2), dict(Y=P + 2), dict(weight=P + 2), dict(bias=P + 2),
        dict(mean=P + 2), dict(rstd=P + 2)))
    st, need = tge.gemm_norm_workspace_bytes(h)
    assert st == OK and need > 0
    good = dict(plan=h, dY=P, X=P, weight=P, mean=P, rstd=P, C=None, dX=P, dweight=P, dbias=P, beta=0.0,
                workspace=P, workspace_bytes=need, stream=None)
    refused(tge.gemm_norm_grad_run, good, (
        dict(plan=None), dict(dY=None), dict(X=None), dict(mean=None), dict(rstd=None), dict(dX=None), dict(beta=1.0),
        dict(beta=NAN), dict(beta=1.0, C=P + 2), dict(workspace=None), dict(workspace=P + 2),
        dict(workspace_bytes=need - 1), dict(dbias=None, workspace=None), dict(dweight=P + 2), dict(dbias=P + 2),
        dict(weight=P + 2), dict(mean=P + 1), dict(rstd=P + 1), dict(dX=P + 1), dict(dY=P + 1), dict(X=P + 1)))
    tge.gemm_norm_plan_destroy(h)
    for kw in (dict(rows=0), dict(N=0)):
        st, e = norm_plan(**kw)
        assert st == OK and tge.gemm_norm_workspace_bytes(e) == (OK, 0)
        assert tge.gemm_norm_run(e, None, None, None, None, None, None, None) == OK
        assert tge.gemm_norm_grad_run(e, None, None, None, None, None, None, None, None, None, 0.0, None, 0, None) == OK
        tge.gemm_norm_plan_destroy(e)


def test_route_run_refusals():
    names = ("logits", "index", "weight", "order", "place", "offsets")
    _, h = route_plan(rows=5000)
    st, need = tge.gemm_route_workspace_bytes(h)
    assert st == OK and need > 0
    good = dict(plan=h, mask=None, slope=P, loss=P, workspace=P, workspace_bytes=need, stream=None, **dict.fromkeys(names, P))
    refused(tge.gemm_route_run, good, [dict(plan=None)] + [{n: None} for n in names] + [
        {n: P + 2} for n in names + ("slope", "loss", "workspace")] + [dict(workspace=None), dict(workspace_bytes=need - 1),
                                                                      dict(workspace_bytes=0)])
    good = dict(plan=h, logits=P, mask=None, index=P, dweight=P, slope=P, dloss=P, dlogits=P, stream=None)
    refused(tge.gemm_route_grad_run, good, (
        dict(plan=None), dict(logits=None), dict(dlogits=None), dict(index=None), dict(slope=None),
        *({n: P + 1} for n in ("logits", "index", "dweight", "slope", "dloss", "dlogits"))))
    tge.gemm_route_plan_destroy(h)
    st, e = route_plan(rows=0)
    assert st == OK and tge.gemm_route_workspace_bytes(e) == (OK, 0)
    assert tge.gemm_route_grad_run(e, None, None, None, None, None, None, None, None) == OK
    # without rows the offsets are still written
    assert tge.gemm_route_run(e, None, None, None, None, None, None, None, None, None, None, 0, None) == INVALID
    tge.gemm_route_plan_destroy(e)


def _kernel(plan):
    return plan.describe().split(" ")[3]


def test_layer_kernel_choice():
    L = tge.LayerPlan
    assert _kernel(L(1, 16384, 4096)) == "layer_rows_16x64"
    assert _kernel(L(16, 4096, 4096)) == "layer_rows_16x16"
    assert _kernel(L(64, 4096, 16384)) == "layer_rows_16x64"
    assert _kernel(L(64, 16384, 4096)) == "layer_rows_64x64"
    assert _kernel(L(64, 16384, 4096, op_b="N")) == "layer_rows_64x64"
    assert _kernel(L(1, 1024, 4096, op_b="N")) == "layer_rows_16x32"
    assert _kernel(L(256, 4096, 4096)) == "layer_rows_64x64"
    assert _kernel(L(512, 4096, 4096)).startswith("gemm_fast")
    assert _kernel(L(8192, 16384, 4096)) == "gemm_fast_256x256"
    assert _kernel(L(5120, 4096, 4096)) == "gemm_fast_128x128"
    assert _kernel(L(1000, 1000, 1000, 4)) == "gemm_fast_64x64"
    assert _kernel(L(3001, 777, 1001, 7, "N", cd="f32")) == "gemm_fast_64x64_rs"
    assert _kernel(L(30000, 4095, 4096, 8, "N")) == "gemm_fast_128x128_rs"
    assert _kernel(L(8, 1024, 2048, 16)).startswith("layer_rows_16x")
    assert _kernel(L(64, 2048, 4096, 64)).startswith("layer_rows_16x")
    f = dict(ab="f32", cd="f32")
    assert _kernel(L(64, 1024, 8192, **f)) == "layer_rows_16x16"
    assert _kernel(L(128, 4096, 4096, **f)) == "layer_rows_32x64"
    assert _kernel(L(256, 4096, 4096, **f)) == "gemm_fast_64x64"
    assert _kernel(L(2048, 4096, 4096, **f)) == "gemm_fast_128x128"
    assert _kernel(L(2048, 4095, 4095, **f)) == "gemm_fast_128x128_rs"
    assert _kernel(L(300, 8191, 511, **f)) == "gemm_fast_64x64_rs"
    assert _kernel(L(8, 1024, 2048, 16, **f)).startswith("layer_rows_16x")
    assert _kernel(L(64, 64, 7)) == "gemm_fast_64x64_rs"
    # sums and rows too short for whole loads, and pinned kernels whose preconditions do not hold: the
    # general one
    for p in (L(64, 7, 64, op_b="N", algo="skinny"), L(64, 3, 3, **f), L(64, 64, 0), L(64, 64, 0, **f),
              L(64, 64, 7, algo="fast"), L(64, 64, 30, algo="fast", **f)):
        assert _kernel(p).startswith("gemm_mfma"), p.describe()


def test_layer_grid_covers_every_split_of_the_rows():
    # the launch is sized from rows and groups alone: no split of the rows may need more tiles
    rng = random.Random(4)
    for _ in range(300):
        E, T, N = rng.randint(1, 90), rng.randint(1, 3000), rng.randint(1, 600)
        algo, tile = rng.choice([("fast", 128), ("fast", 256), ("skinny", 0), ("skinny", 64), ("general", 64), ("auto", 0)])
        ab = rng.choice(["f16", "f32"])
        p = tge.LayerPlan(T, N, 64, E, "T", ab=ab, cd=ab, algo=algo, tile=tile)
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


@pytest.mark.parametrize("type, es", [("f32", 4), ("f16", 2), ("bf16", 2)])
def test_norm_teams_hold_every_row(type, es):
    # waves * chunks pieces of 1 KiB hold a row, of at most 16 waves; the workspace is a partial sum of both
    # gradients per workgroup, within what is documented
    for n in (1, 2, 511, 512, 513, 1000, 2049, 4096, 5000, 8193, 10000, 65536 // es):
        for rows in (1, 7, 5000, 1 << 20):
            p = tge.NormPlan(rows, n, type)
            waves, chunks, grid, grad = map(int, re.search(r"waves (\d+) chunks (\d+) grid (\d+), gradient (\d+)", p.describe()).groups())
            assert waves in (1, 2, 3, 4, 6, 8, 12, 16) and waves * chunks * 1024 >= n * es
            assert p.workspace_bytes == grad * 2 * n * 4 <= (2 << 20) * -(-n // 1024) and 1 <= grid <= rows


def test_route_blocks_cover_every_row():
    rng = random.Random(5)
    for _ in range(200):
        experts, rows = rng.randint(1, 1024), rng.choice([0, 1, rng.randint(1, 500), rng.randint(1, 1 << 20)])
        p = tge.RoutePlan(rows, experts, min(experts, rng.randint(1, 16)))
        lanes, per, blocks, each = map(int, re.search(r"lanes (\d+) x (\d+) blocks (\d+) of (\d+)", p.describe()).groups())
        assert lanes * per >= experts and blocks * each >= rows and (blocks - 1) * each <= max(rows - 1, 0) and blocks <= 256
        side = max(4, 1 << (blocks - 1).bit_length())
        assert p.workspace_bytes == ((2 * experts + 1) * side * 4 if blocks > 1 else 0)


def test_binding_checks():
    f16, i32, u8 = torch.float16, torch.int32, torch.uint8
    p = tge.LayerPlan(10, 8, 16, 3, "N", ldc=12, cd="f32", act="silu")
    for what, t in (("A", torch.zeros(10, 16, dtype=f16)), ("B", torch.zeros(3, 16, 8, dtype=f16)), ("D", torch.zeros(10, 12)),
                    ("pre", torch.zeros(9 * 12 + 8)), ("bias", torch.zeros(3, 8)), ("offsets", torch.zeros(4, dtype=i32))):
        p.check(what, t)
    for what, t, err in (("A", torch.zeros(10, 16), TypeError), ("A", torch.zeros(9, 16, dtype=f16), ValueError),
                         ("A", torch.zeros(16, 10, dtype=f16).t(), ValueError), ("pre", torch.zeros(10, 12, dtype=f16), TypeError),
                         ("B", torch.zeros(2, 16, 8, dtype=f16), ValueError), ("D", torch.zeros(10, 8), ValueError),
                         ("pre", torch.zeros(10, 8), ValueError), ("bias", torch.zeros(23), ValueError),
                         ("bias", torch.zeros(24, dtype=f16), TypeError), ("offsets", torch.zeros(3, dtype=i32), ValueError),
                         ("offsets", torch.zeros(4, dtype=torch.int64), TypeError)):
        with pytest.raises(err):
            p.check(what, t)
    n = tge.NormPlan(10, 8, "f16", ldx=9)
    for what, t in (("X", torch.zeros(10, 9, dtype=f16)), ("dX", torch.zeros(10, 9, dtype=f16)), ("Y", torch.zeros(10, 8, dtype=f16)),
                    ("weight", torch.zeros(8)), ("mean", torch.zeros(10)), ("workspace", torch.zeros(n.workspace_bytes, dtype=u8))):
        n.check(what, t)
    for what, t, err in (("X", torch.zeros(10, 8, dtype=f16), ValueError), ("X", torch.zeros(10, 9), TypeError),
                         ("Y", torch.zeros(9, 8, dtype=f16), ValueError), ("weight", torch.zeros(8, dtype=f16), TypeError),
                         ("weight", torch.zeros(7), ValueError), ("rstd", torch.zeros(9), ValueError),
                         ("dbias", torch.zeros(7), ValueError), ("workspace", torch.zeros(n.workspace_bytes - 1, dtype=u8), ValueError),
                         ("workspace", torch.zeros(n.workspace_bytes), TypeError)):
        with pytest.raises(err):
            n.check(what, t)
    r = tge.RoutePlan(3000, 10, 2, "f32", ldl=12)
    for what, t in (("logits", torch.zeros(3000, 12)), ("index", torch.zeros(3000, 2, dtype=i32)), ("weight", torch.zeros(3000, 2)),
                    ("mask", torch.zeros(3000, dtype=u8)), ("offsets", torch.zeros(11, dtype=i32)), ("loss", torch.zeros(1)),
                    ("workspace", torch.zeros(r.workspace_bytes, dtype=u8))):
        r.check(what, t)
    for what, t, err in (("logits", torch.zeros(3000, 10), ValueError), ("logits", torch.zeros(3000, 12, dtype=f16), TypeError),
                         ("index", torch.zeros(3000, 2, dtype=torch.int64), TypeError), ("order", torch.zeros(5999, dtype=i32), ValueError),
                         ("mask", torch.zeros(3000, dtype=torch.bool), TypeError), ("mask", torch.zeros(2999, dtype=u8), ValueError),
                         ("offsets", torch.zeros(10, dtype=i32), ValueError), ("slope", torch.zeros(9), ValueError),
                         ("loss", torch.zeros(0), ValueError), ("workspace", torch.zeros(r.workspace_bytes - 1, dtype=u8), ValueError)):
        with pytest.raises(err):
            r.check(what, t)
    for cls, args in ((tge.LayerPlan, (10, 8, 16, 0)), (tge.NormPlan, (10, 8, "i8")), (tge.NormPlan, (-1, 8)),
                      (tge.RoutePlan, (10, 8, 9)), (tge.RoutePlan, (10, 2000, 2))):
        with pytest.raises(tge.GemmError):
            cls(*args)


def test_operands_checked_together():
    # the module gives pointers for what passes as it is, and nothing where a tensor does not fit (the checks
    # one by one then name it)
    from tiled_gemm_epilogues_amd import _operands
    p = tge.NormPlan(4, 8, "f32")
    assert tuple(p._pointers(0, 1, None, 3, 4, 5, 6)) == (1, None, 3, 4, 5, 6)
    for what, args in (("X", (torch.zeros(4, 8), None, None, None, None, None)), ("rstd", (1, None, None, 4, 5, torch.zeros(4)))):
        with pytest.raises(ValueError, match=f"{what} must be a device tensor"):
            p._pointers(0, *args)
    one = _operands.Operands(((torch.float32, 4, 2),))
    assert one(0, None) == (None,) and one(0, 7) == (7,)
    for t in (torch.zeros(2, 2), "no tensor", torch.zeros(2, 2, device="meta")):
        assert one(0, t) is None
    for bad in (lambda: _operands.Operands(1), lambda: _operands.Operands(((1, 2, 3),)),
                lambda: _operands.Operands(((torch.float32, 2, "x"),)), lambda: one(0), lambda: one(0, 1, 2), lambda: one("x", 1),
                lambda: one(0, t=1)):
        with pytest.raises(TypeError):
            bad()
