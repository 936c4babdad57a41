"""A layer's products (bias, activation, residual, kept argument, gradient) against 64 bits, over every
kernel, type, layout, activation, odd sizes, strides and row ranges.  The sums are exact (integers
times a power of two), so that what is compared is the epilogue; accumulation errors have their own
test."""
import numpy as np
import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import SENTINEL, TORCH_DT, ints, offsets_of
from layer_helpers import ACTS, U, act64, act_bound, close, rounding, slope64, slope_bound

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")
PAIRS = [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]
KERNELS = [("general", 64), ("general", 128), ("fast", 64), ("fast", 128), ("fast", 256), ("staged", 64),
           ("staged", 128), ("skinny", 64), ("skinny", 16)]
NAMES = {"general": "gemm_mfma", "fast": "gemm_fast", "staged": "_rs", "skinny": "layer_rows"}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tile_of(algo, tile, op_b):
    return 32 if algo == "skinny" and tile == 16 and op_b == "N" else tile


class Problem:
    """Operands with exact sums, z = alpha * (A B) + bias within about -12 .. 12, and D's start."""

    def __init__(self, seed, rows, N, K, op_b, ab, cd, groups=1, counts=None, pad=(0, 0, 0), share_bias=False):
        g = np.random.default_rng(seed)
        tab, tcd = TORCH_DT[ab], TORCH_DT[cd]
        self.rows, self.N, self.K, self.op_b, self.ab, self.cd, self.groups = rows, N, K, op_b, ab, cd, groups
        self.alpha = 0.125
        b_rows, b_cols = (K, N) if op_b == "N" else (N, K)
        self.lda, self.ldb, self.ldc = K + pad[0], b_cols + pad[1], N + pad[2]
        keep = min(1.0, 500.0 / max(K, 1))
        self.A = ints(g, (rows, self.lda), -3, 3, tab) * torch.from_numpy(g.random((rows, self.lda)) < keep)
        self.B = ints(g, (groups, b_rows, self.ldb), -2, 2, tab)
        self.bias = ints(g, (1 if share_bias else groups, N), -16, 16, torch.float32) / 8
        self.stride_bias = 0 if share_bias else N
        self.C = (ints(g, (rows, self.ldc), -40, 40, torch.float32) / 8).to(tcd)
        self.Zin = (ints(g, (rows, self.ldc), -60, 60, torch.float32) / 8).to(tcd)
        self.offs = offsets_of(counts, 1) if counts is not None else None

    def plan(self, act, algo="auto", tile=0):
        return tge.LayerPlan(self.rows, self.N, self.K, self.groups, self.op_b, self.lda, self.ldb, self.ldc,
                             stride_bias=self.stride_bias, ab=self.ab, cd=self.cd, act=act, algo=algo, tile=tile)

    def ranges(self):
        if self.offs is None:
            return [(0, 0, self.rows)]
        return [(e, lo, hi) for e, (lo, hi) in enumerate(zip(self.offs[:-1], self.offs[1:])) if lo < hi]

    def product(self):
        """alpha * A B of the rows in the ranges, zero elsewhere, in 64 bits; and which rows they are."""
        z = torch.zeros(self.rows, self.N, dtype=torch.float64)
        used = torch.zeros(self.rows, dtype=torch.bool)
        for e, lo, hi in self.ranges():
            b = self.B[e].double()
            b = b[:, :self.N] if self.op_b == "N" else b[:, :self.K].t()
            z[lo:hi] = self.alpha * (self.A[lo:hi, :self.K].double() @ b)
            used[lo:hi] = True
        return z, used

    def biases(self):
        full = torch.zeros(self.rows, self.N, dtype=torch.float64)
        for e, lo, hi in self.ranges():
            full[lo:hi] = self.bias[min(e, len(self.bias) - 1)].double()
        return full

    def device(self):
        d = None if self.offs is None else torch.from_numpy(self.offs).to(DEV)
        return self.A.to(DEV), self.B.to(DEV), self.C.to(DEV), self.bias.to(DEV), d

    def fresh(self):
        return torch.full((self.rows, self.ldc), SENTINEL, dtype=TORCH_DT[self.cd], device=DEV)


def untouched(p, used, *outs):
    for t in outs:
        t = t.cpu().double()
        assert (t[:, p.N:] == SENTINEL).all(), "between the rows"
        assert (t[~used] == SENTINEL).all(), "rows outside the ranges"


def check_forward(p, act, plan, bias=True, residual=True, pre=True, in_place=False):
    A, B, C, b, offs = p.device()
    D, Z = p.fresh(), p.fresh()
    beta = -0.5
    if in_place:
        D = C.clone()
        D[:, p.N:] = SENTINEL
    prod, used = p.product()
    if in_place:
        D[~used.to(DEV)] = SENTINEL
    plan.run(A, B, (D if in_place else C) if residual else None, D, offs, b if bias else None, Z if pre else None,
             alpha=p.alpha, beta=beta if residual else 0.0)
    z = prod + (p.biases() if bias else 0.0)
    tcd = TORCH_DT[p.cd]
    act_z = act64(act, z)
    want = act_z + (beta * p.C[:, :p.N].double() if residual else 0.0)
    bound = act_bound(act, z, tcd) + (U * want.abs() if residual else 0.0)
    bound = bound + rounding(want.abs() + bound, tcd) * 1.0001
    close(D[:, :p.N][used.to(DEV)], want[used], bound[used], f"{act} D")
    untouched(p, used, D)
    if pre:
        close(Z[:, :p.N][used.to(DEV)], z[used], (rounding(z, tcd) if p.cd != "f32" else torch.zeros_like(z))[used], f"{act} Z")
        untouched(p, used, Z)
    else:
        assert (Z.cpu().double() == SENTINEL).all()


def check_grad(p, act, plan, in_place=False):
    A, B, _, _, offs = p.device()
    Zin = p.Zin.to(DEV)
    prod, used = p.product()
    D = p.fresh()
    if in_place:
        Zin[:, p.N:] = SENTINEL
        Zin[~used.to(DEV)] = SENTINEL
        D = Zin
    plan.run_grad(A, B, Zin, D, offs, alpha=p.alpha)
    z, tcd = p.Zin[:, :p.N].double(), TORCH_DT[p.cd]
    want = prod * slope64(act, z)
    bound = prod.abs() * slope_bound(act, z, tcd) + U * want.abs()
    bound = bound + rounding(want.abs() + bound, tcd) * 1.0001
    close(D[:, :p.N][used.to(DEV)], want[used], bound[used], f"{act} gradient")
    untouched(p, used, D)


@pytest.mark.parametrize("ab,cd", PAIRS + [("f32", "f32")])
@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_every_kernel(algo, tile, op_b, ab, cd):
    # whole tiles and ragged ones on both edges; K with a tail
    for i, (rows, N, K) in enumerate([(256, 256, 128), (300, 328, 200), (37, 72, 72)]):
        p = Problem(i, rows, N, K, op_b, ab, cd)
        for act in ACTS:
            plan = p.plan(act, algo, tile_of(algo, tile, op_b))
            assert NAMES[algo] in plan.describe(), plan.describe()
            check_forward(p, act, plan)
            check_grad(p, act, plan)
        check_forward(p, "gelu", p.plan("gelu", algo, tile_of(algo, tile, op_b)), bias=False, residual=False, pre=False)


@pytest.mark.parametrize("ab,cd", PAIRS + [("f32", "f32")])
@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_ranges_in_every_kernel(algo, tile, op_b, ab, cd):
    # experts without rows, with one, and with more than a tile; rows in front and behind
    p = Problem(7, 420, 136, 136, op_b, ab, cd, groups=6, counts=[3, 0, 270, 1, 0, 140], pad=(8, 16, 8))
    for act in ("silu", "gelu", "none"):
        plan = p.plan(act, algo, tile_of(algo, tile, op_b))
        check_forward(p, act, plan)
        check_grad(p, act, plan)


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("algo,tile", [k for k in KERNELS if k[0] != "fast"])
def test_fp32(algo, tile, op_b):
    tile = tile_of(algo, tile, op_b)
    for i, (rows, N, K, groups, counts) in enumerate([(130, 140, 70, 1, None), (1, 1, 1, 1, None),
                                                      (90, 33, 35, 4, [0, 50, 2, 30]), (17, 65, 4, 1, None),
                                                      (48, 70, 300, 3, [3, 20, 24]), (28, 64, 1001, 2, [10, 17])]):
        p = Problem(20 + i, rows, N, K, op_b, "f32", "f32", groups, counts, pad=(1, 3, 5))
        for act in ACTS:
            plan = p.plan(act, algo, tile)
            assert K == 1 or NAMES[algo] in plan.describe(), plan.describe()
            check_forward(p, act, plan)
            check_grad(p, act, plan)


@pytest.mark.parametrize("rows", [1, 2, 15, 17, 64, 129, 513])
@pytest.mark.parametrize("N,K", [(1, 8), (7, 9), (8, 64), (65, 1), (129, 1001), (264, 65)])
def test_odd_sizes_choose_their_kernel(rows, N, K):
    for ab, cd, op_b in (("bf16", "bf16", "T"), ("f16", "f32", "N")):
        p = Problem(rows * 1000 + N, rows, N, K, op_b, ab, cd, pad=(1, 1, 3))
        check_forward(p, "gelu_tanh", p.plan("gelu_tanh"))
        check_grad(p, "silu", p.plan("silu"))


@pytest.mark.parametrize("off", [1, 3])
def test_operands_off_the_16_byte_grid(off):
    # pointers that are aligned to the element only, in a plan whose leading dimensions are whole chunks
    p = Problem(31, 200, 192, 128, "T", "bf16", "bf16", pad=(0, 0, 0))
    plan = p.plan("silu")

    def moved(t):
        buf = torch.full((t.numel() + off,), NAN, dtype=t.dtype, device=DEV)
        buf[off:] = t.reshape(-1).to(DEV)
        return buf[off:].view(t.shape)
    prod, _ = p.product()
    z = prod + p.biases()
    for which in range(4):
        ops = [p.A, p.B, p.C, p.fresh()]
        ops = [moved(t) if i == which else t.to(DEV) for i, t in enumerate(ops)]
        plan.run(ops[0], ops[1], ops[2], ops[3], None, p.bias.to(DEV), alpha=p.alpha, beta=1.0)
        want = act64("silu", z) + p.C.double()
        bound = act_bound("silu", z, torch.bfloat16) + U * want.abs()
        close(ops[3], want, bound + rounding(want.abs() + bound, torch.bfloat16) * 1.0001)


@pytest.mark.parametrize("algo,tile", KERNELS)
def test_in_place(algo, tile):
    # C == D forward, Z == D in the gradient
    p = Problem(41, 300, 200, 128, "T", "bf16", "bf16")
    plan = p.plan("gelu", algo, tile)
    check_forward(p, "gelu", plan, in_place=True)
    check_grad(p, "gelu", plan, in_place=True)
    p = Problem(42, 300, 200, 128, "T", "f16", "f32", groups=3, counts=[100, 7, 150])
    check_forward(p, "silu", p.plan("silu", algo, tile), in_place=True)
    check_grad(p, "silu", p.plan("silu", algo, tile), in_place=True)


def test_shared_weights_and_bias():
    p = Problem(51, 200, 96, 64, "T", "f16", "f16", groups=3, counts=[60, 70, 60], share_bias=True)
    check_forward(p, "relu", p.plan("relu"))


def test_empty_problems():
    z = torch.zeros
    for rows, N, K in ((0, 8, 8), (8, 0, 8)):
        plan = tge.LayerPlan(rows, N, K, ab="f16", cd="f16", act="gelu")
        plan.run(z(rows, K, dtype=torch.float16, device=DEV), z(N, K, dtype=torch.float16, device=DEV), None,
                 z(rows, N, dtype=torch.float16, device=DEV))
    # K == 0: D = act(bias) + beta * C
    plan = tge.LayerPlan(5, 9, 0, ab="f16", cd="f32", act="silu")
    b = torch.arange(-4, 5, device=DEV, dtype=torch.float32)
    C, D = torch.ones(5, 9, device=DEV), torch.full((5, 9), NAN, device=DEV)
    plan.run(None, None, C, D, None, b, beta=2.0)
    v = b.double().cpu().expand(5, 9)
    close(D, act64("silu", v) + 2, act_bound("silu", v, torch.float32) + 4 * U)
    # a range that holds no row leaves everything
    plan = tge.LayerPlan(5, 16, 8, 3, "T", ab="f16", cd="f16", act="silu")
    D = torch.full((5, 16), SENTINEL, dtype=torch.float16, device=DEV)
    plan.run(z(5, 8, dtype=torch.float16, device=DEV), z(3, 16, 8, dtype=torch.float16, device=DEV), None, D,
             z(4, dtype=torch.int32, device=DEV))
    assert (D == SENTINEL).all()


@pytest.mark.parametrize("offs", [[5, 3, 40, 20], [-7, 10, 90, 30], [0, 2 ** 31 - 1, 3, -2 ** 31]])
def test_offsets_out_of_order_stay_inside(offs):
    # their values are undefined; the operands' surroundings are not touched
    rows, N, K = 50, 72, 64
    for algo, tile in KERNELS:
        plan = tge.LayerPlan(rows, N, K, 3, "T", ab="f16", cd="f16", act="gelu", algo=algo, tile=tile)
        A = torch.zeros(rows, K, dtype=torch.float16, device=DEV)
        B = torch.zeros(3, N, K, dtype=torch.float16, device=DEV)
        around = torch.full((3, rows, N), SENTINEL, dtype=torch.float16, device=DEV)
        Z = torch.full((3, rows, N), SENTINEL, dtype=torch.float16, device=DEV)
        plan.run(A, B, None, around[1], torch.tensor(offs, dtype=torch.int64).to(torch.int32).to(DEV), None, Z[1])
        assert (around[[0, 2]] == SENTINEL).all() and (Z[[0, 2]] == SENTINEL).all()


@pytest.mark.parametrize("algo,tile", [("general", 64), ("fast", 64), ("staged", 64), ("skinny", 64)])
def test_extreme_arguments(algo, tile):
    # z from the smallest to the largest: one column of B picks the row's value; fp32 results
    vals = [0.0, -0.0, 1e-7, -1e-7, 0.75, -0.75, 5.0, -5.0, 9.0, -9.0, 14.0, -14.0, 100.0, -100.0, 65504.0, -65504.0]
    rows, N, K = 16, 64, 64
    A = torch.zeros(rows, K, dtype=torch.float16)
    A[:, 0] = torch.tensor(vals, dtype=torch.float16)
    B = torch.zeros(N, K, dtype=torch.float16)
    B[:, 0] = 1
    z = A[:, :1].double().expand(rows, N)
    for act in ACTS:
        plan = tge.LayerPlan(rows, N, K, ab="f16", cd="f32", act=act, algo=algo, tile=tile)
        D = torch.full((rows, N), NAN, device=DEV)
        plan.run(A.to(DEV), B.to(DEV), None, D)
        want = act64(act, z)
        close(D, want, act_bound(act, z, torch.float32) + U * want.abs(), act)
        ones = torch.zeros(rows, K, dtype=torch.float16, device=DEV)
        ones[:, 0] = 1
        plan.run_grad(ones, B.to(DEV), z.float().contiguous().to(DEV), D)
        close(D, slope64(act, z), slope_bound(act, z, torch.float32) + U, act + " slope")


@pytest.mark.parametrize("algo,tile", KERNELS)
def test_nan_and_infinities_keep_to_their_rows(algo, tile):
    rows, N, K = 40, 80, 64
    g = np.random.default_rng(3)
    A = ints(g, (rows, K), -2, 2, torch.float16)
    A[3, 5], A[7, 0], A[39, 63] = NAN, float("inf"), NAN
    B = ints(g, (N, K), 1, 3, torch.float16) / 16
    z = A.double() @ B.double().t()
    for act in ACTS:
        plan = tge.LayerPlan(rows, N, K, ab="f16", cd="f16", act=act, algo=algo, tile=tile)
        D, Z = (torch.zeros(rows, N, dtype=torch.float16, device=DEV) for _ in range(2))
        plan.run(A.to(DEV), B.to(DEV), None, D, None, None, Z)
        bad = torch.zeros(rows, dtype=torch.bool)
        bad[[3, 39]] = True
        got = D.cpu().double()
        assert got[bad].isnan().all() and Z.cpu()[bad].isnan().all()
        assert (got[7] == float("inf")).all()
        bad[7] = True
        assert got[~bad].isfinite().all()
        want = act64(act, z[~bad])
        bound = act_bound(act, z[~bad], torch.float16)
        close(got[~bad], want, bound + rounding(want.abs() + bound, torch.float16) * 1.0001, act)


@pytest.mark.parametrize("ab,cd", PAIRS + [("f32", "f32")])
def test_accumulation(ab, cd):
    # random values: K products and K - 1 additions of fp32 (each at most one step, 2 U, of the sum of the
    # terms' sizes), through an activation that moves its argument's error by at most 1.13
    g = torch.Generator().manual_seed(9)
    for rows, N, K in ((500, 392, 1000), (9, 512, 4096)):
        A = torch.randn(rows, K, generator=g).to(TORCH_DT[ab])
        B = (torch.randn(N, K, generator=g) * K ** -0.5).to(TORCH_DT[ab])
        bias = torch.randn(N, generator=g)
        z = A.double() @ B.double().t() + bias.double()
        mag = A.double().abs() @ B.double().abs().t() + bias.double().abs()
        dz = (2 * K + 2) * U * mag
        plan = tge.LayerPlan(rows, N, K, ab=ab, cd=cd, act="gelu")
        D, Z = (torch.zeros(rows, N, dtype=TORCH_DT[cd], device=DEV) for _ in range(2))
        plan.run(A.to(DEV), B.to(DEV), None, D, None, bias.to(DEV), Z)
        close(Z, z, dz + rounding(z.abs() + dz, TORCH_DT[cd]) * 1.0001)
        want = act64("gelu", z)
        bound = 1.13 * dz + act_bound("gelu", z, TORCH_DT[cd]) * 1.01
        close(D, want, bound + rounding(want.abs() + bound, TORCH_DT[cd]) * 1.0001)


def test_slopes_are_the_forward_passes_differences():
    # fp32, identity weights: (D(z + h) - D(z - h)) / 2h is the slope up to h^2 / 6 of the third
    # derivative (at most 2.5 in size) and the roundings of D over 2h
    n = 96
    z = torch.linspace(-6, 6, n).expand(8, n).contiguous().to(DEV)
    eye, h = torch.eye(n, device=DEV), 2.0 ** -6
    for act in ("gelu", "gelu_tanh", "silu"):
        plan = tge.LayerPlan(8, n, n, ab="f32", cd="f32", act=act)
        up, down, slope = (torch.zeros(8, n, device=DEV) for _ in range(3))
        plan.run(z + h, eye, None, up)
        plan.run(z - h, eye, None, down)
        plan.run_grad(torch.ones(8, n, device=DEV), eye, z, slope)
        diff = (up.double() - down.double()) / (2 * h)
        bound = 2.5 * h * h / 6 + (7 * 100 * U) / h + torch.zeros_like(diff.cpu())
        close(slope, diff.cpu(), bound, act)


def test_runs_repeat_and_graphs_follow_offsets():
    p = Problem(61, 300, 136, 128, "T", "bf16", "bf16", groups=4, counts=[100, 0, 150, 40])
    plan = p.plan("gelu")
    A, B, C, b, offs = p.device()
    D, Z, G = p.fresh(), p.fresh(), p.fresh()

    def step():
        plan.run(A, B, C, D, offs, b, Z, alpha=p.alpha, beta=1.0)
        plan.run_grad(A, B, Z, G, offs, alpha=p.alpha)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in ([100, 0, 150, 40], [0, 290, 0, 1], [73, 73, 73, 73], [0, 0, 0, 0]):
        offs.copy_(torch.from_numpy(offsets_of(counts, 1)))
        for t in (D, Z, G):
            t.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (D, Z, G)]
        for t in (D, Z, G):
            t.fill_(SENTINEL)
        step()
        for x, y in zip(got, (D, Z, G)):
            assert torch.equal(x, y)


def test_two_streams_share_a_plan():
    p = Problem(71, 260, 256, 128, "T", "f16", "f16")
    plan = p.plan("silu")
    A, B, C, b, _ = p.device()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [p.fresh() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, D in zip(streams, outs):
            plan.run(A, B, C, D, None, b, alpha=p.alpha, beta=1.0, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    D = p.fresh()
    plan.run(A, B, C, D, None, b, alpha=p.alpha, beta=1.0)
    assert torch.equal(D, outs[0])


def test_weights_past_the_caches():
    # few rows of weights of 128 MiB and more: read without the caches, in every shape of the kernel, whole
    # chunks and a rest, and by expert; the sums are exact
    for rows, N, K, groups, counts in ((1, 16400, 4104, 1, None), (17, 4100, 16400, 1, None), (60, 16400, 4104, 1, None),
                                       (40, 2056, 4160, 8, [3, 0, 9, 1, 8, 8, 0, 10])):
        p = Problem(N + rows, rows, N, K, "T", "bf16", "bf16", groups=groups, counts=counts)
        plan = p.plan("silu")
        assert "layer_rows" in plan.describe() and groups * N * K * 2 >= 128 << 20
        check_forward(p, "silu", plan)


def test_refusals_name_the_operand():
    plan = tge.LayerPlan(8, 16, 16, act="gelu")
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device=DEV)
    A, B, D = z(8, 16), z(16, 16), z(8, 16)
    for args, err in (((A.cpu(), B, None, D), "A must be a device tensor"), ((A, B[:15], None, D), "B holds"),
                      ((A, B, None, D[:7]), "D holds")):
        with pytest.raises(ValueError, match=err):
            plan.run(*args)
    with pytest.raises(TypeError, match="pre must be"):
        plan.run(A, B, None, D, pre=D.float())
    for call in (lambda: plan.run(A, B, None, D, beta=1.0), lambda: plan.run(A, B, None, D, pre=D),
                 lambda: plan.run(A, B, D, z(8, 16), pre=D, beta=1.0), lambda: plan.run_grad(A, B, None, D),
                 lambda: plan.run(A, B, None, D, alpha=NAN),
                 lambda: tge.LayerPlan(8, 16, 16, 2).run(A, z(2, 16, 16), None, D)):
        with pytest.raises(tge.GemmError, match="INVALID_VALUE"):
            call()


def test_offsets_beyond_32_bits():
    # D of more than 2^32 bytes: the last rows are where they belong
    rows, N, K = 300000, 8192, 64
    A = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    A[-1, 0], A[0, 0] = 3, 2
    B = torch.zeros(N, K, dtype=torch.bfloat16, device=DEV)
    B[:, 0] = 1
    D = torch.full((rows, N), SENTINEL, dtype=torch.bfloat16, device=DEV)
    C = torch.ones(rows, N, dtype=torch.bfloat16, device=DEV)
    plan = tge.LayerPlan(rows, N, K, ab="bf16", cd="bf16", act="relu")
    plan.run(A, B, C, D, beta=1.0)
    assert (D[0] == 3).all() and (D[-1] == 4).all() and (D[1:-1:997] == 1).all()
