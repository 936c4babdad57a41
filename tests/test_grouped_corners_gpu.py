"""Calls of the grouped and 4-bit plans at the edge of what their documentation allows: offsets out of
order and out of bounds (with more than one scan of 64 ranges), operands off the 16-byte grid in plans
that choose their own kernel, biases shared by all experts, and NaN where a gate is closed."""
import numpy as np
import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import SENTINEL, TORCH_DT, grad_reference, ints, offsets_of, rounded, rows_reference
from test_quant_gpu import dequantised

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def guarded(n, dtype):
    """A buffer of sentinels with n elements in its middle."""
    buf = torch.full((n + 8192,), SENTINEL, dtype=dtype, device=DEV)
    return buf, buf[4096:4096 + n]


def untouched(buf, n):
    out = buf.cpu()
    return bool((out[:4096] == SENTINEL).all() and (out[4096 + n:] == SENTINEL).all())


def bad_offsets(groups, rows, seed):
    """Offsets that are neither ordered nor within [0, rows]."""
    g = np.random.default_rng(seed)
    o = g.integers(-2 * rows, 3 * rows, groups + 1)
    o[g.integers(0, groups + 1, 3)] = [2 ** 31 - 1, -2 ** 31, rows]
    return torch.from_numpy(o.astype(np.int32)).to(DEV)


@pytest.mark.parametrize("groups", [4, 150])
@pytest.mark.parametrize("algo,tile", [("auto", 0), ("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128),
                                       ("staged", 64), ("general", 128), ("general", 64)])
def test_gradients_of_bad_offsets_stay_inside(groups, algo, tile):
    # undefined values, but every access stays inside the operands: the gradients' own elements are all
    # written (with sums of finite values), and nothing around them
    T, M, N = 100, 72, 64
    A = torch.ones(T, M, dtype=torch.float16, device=DEV)
    B = torch.ones(T, N, dtype=torch.float16, device=DEV)
    for seed in range(3):
        buf, D = guarded(groups * M * N, torch.float32)
        sbuf, sums = guarded(groups * N, torch.float32)
        D.fill_(NAN), sums.fill_(NAN)
        tge.GroupedGradPlan(T, M, N, groups, algo=algo, tile=tile).run(A, B, None, D, bad_offsets(groups, T, seed), sums)
        assert untouched(buf, D.numel()) and untouched(sbuf, sums.numel())
        assert ((D >= 0) & (D <= T)).all() and ((sums >= 0) & (sums <= T)).all()


@pytest.mark.parametrize("groups", [4, 150])
@pytest.mark.parametrize("algo,tile", [("auto", 0), ("fast", 256), ("fast", 128), ("staged", 64), ("skinny", 0),
                                       ("skinny", 64), ("general", 64)])
def test_rows_of_bad_offsets_stay_inside(groups, algo, tile):
    T, N, K = 100, 72, 64
    A = torch.ones(T, K, dtype=torch.float16, device=DEV)
    B = torch.ones(groups, K, N, dtype=torch.float16, device=DEV)
    for seed in range(3):
        buf, D = guarded(T * N, torch.float16)
        tge.GroupedPlan(T, N, K, groups, algo=algo, tile=tile).run(A, B, None, D, bad_offsets(groups, T, seed))
        assert untouched(buf, D.numel())
        assert ((D == SENTINEL) | (D == K)).all()


@pytest.mark.parametrize("groups", [4, 150])
@pytest.mark.parametrize("algo,tile", [("auto", 0), ("skinny", 16), ("skinny", 64), ("fast", 128)])
def test_quant_of_bad_offsets_stays_inside(groups, algo, tile):
    T, N, K, block = 100, 72, 128, 64
    A = torch.ones(T, K, dtype=torch.bfloat16, device=DEV)
    Q = torch.full((groups, N, K // 2), 0x99, dtype=torch.uint8, device=DEV)
    scales = torch.ones(groups, N, K // block, dtype=torch.bfloat16, device=DEV)
    zeros = torch.full((groups, N, K // block), 8, dtype=torch.uint8, device=DEV)
    for seed in range(3):
        buf, D = guarded(T * N, torch.bfloat16)
        tge.QuantPlan(T, N, K, block, groups, zeros=True, ab="bf16", cd="bf16", algo=algo, tile=tile).run(
            A, Q, scales, zeros, None, D, bad_offsets(groups, T, seed))
        assert untouched(buf, D.numel())
        assert ((D == SENTINEL) | (D == K)).all()


def off(x):
    """x on the device, one element off its allocation."""
    return torch.cat([torch.zeros(1, dtype=x.dtype), x.reshape(-1)]).to(DEV)[1:]


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("counts", [[100, 60], [300, 0, 500]])
@pytest.mark.parametrize("which", ["A", "B", "AB"])
def test_rows_off_the_grid_in_a_plan_of_its_own_choice(op_b, counts, which):
    # leading dimensions of whole chunks, but a pointer between them: the register-staged kernel runs
    g = np.random.default_rng(1)
    T, E, N, K = sum(counts), len(counts), 2048, 512
    A, B = ints(g, (T, K), -2, 2, torch.bfloat16), ints(g, (E, *((K, N) if op_b == "N" else (N, K))), -2, 2, torch.bfloat16)
    offs = offsets_of(counts)
    D = torch.full((T, N), SENTINEL, device=DEV)
    p = tge.GroupedPlan(T, N, K, E, op_b, ab="bf16", cd="f32")
    p.run(off(A) if "A" in which else A.to(DEV), off(B) if "B" in which else B.to(DEV), None, D, torch.from_numpy(offs).to(DEV))
    want = rows_reference(A, B, None, torch.zeros(T, N), offs, op_b, None, 1.0, 0.0, "none")
    assert torch.equal(D.cpu().double(), want)


@pytest.mark.parametrize("M,N,counts", [(1024, 704, [100, 3, 0, 200]), (2048, 2048, [65, 130] + [16] * 6)])
@pytest.mark.parametrize("which", ["A", "B", "AB"])
@pytest.mark.parametrize("algo", ["auto", "fast"])
def test_gradients_off_the_grid(M, N, counts, which, algo):
    g = np.random.default_rng(2)
    T, E = sum(counts), len(counts)
    A, B = ints(g, (T, M), -2, 2, torch.float16), ints(g, (T, N), -2, 2, torch.float16)
    offs = offsets_of(counts)
    D, sums = torch.full((E, M, N), SENTINEL, device=DEV), torch.full((E, N), SENTINEL, device=DEV)
    p = tge.GroupedGradPlan(T, M, N, E, algo=algo)
    assert "gemm_fast" in p.describe() and "_rs" not in p.describe()
    p.run(off(A) if "A" in which else A.to(DEV), off(B) if "B" in which else B.to(DEV), None, D,
          torch.from_numpy(offs).to(DEV), sums)
    want, want_sums = grad_reference(A.float(), B.float(), None, offs, 1.0, 0.0)
    assert torch.equal(D.cpu().double(), want) and torch.equal(sums.cpu().double(), want_sums)


@pytest.mark.parametrize("algo,tile", [("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128), ("skinny", 0),
                                       ("skinny", 64), ("general", 64)])
def test_one_bias_for_all_experts(algo, tile):
    g = np.random.default_rng(3)
    counts, N, K = [40, 0, 150, 3], 136, 64
    A, B = ints(g, (193, K), -3, 3, torch.float16), ints(g, (4, N, K), -3, 3, torch.float16)
    bias, offs = ints(g, (1, N), -9, 9, torch.float32), offsets_of(counts)
    D = torch.empty(193, N, device=DEV)
    tge.GroupedPlan(193, N, K, 4, "T", stride_bias=0, cd="f32", epilogue="bias", algo=algo, tile=tile).run(
        A.to(DEV), B.to(DEV), None, D, torch.from_numpy(offs).to(DEV), bias.to(DEV))
    want = rows_reference(A, B, None, torch.zeros(193, N), offs, "T", bias.expand(4, N), 1.0, 0.0, "bias")
    assert torch.equal(D.cpu().double(), want)


@pytest.mark.parametrize("algo,tile", [("skinny", 16), ("skinny", 64), ("fast", 128)])
def test_one_4bit_bias_for_all_experts(algo, tile):
    g = np.random.default_rng(4)
    counts, N, K = [40, 0, 150, 3], 72, 128
    A = ints(g, (193, K), -3, 3, torch.bfloat16)
    Q = torch.from_numpy(g.integers(0, 256, (4, N, K // 2)).astype(np.uint8))
    scales = torch.ones(4, N, 2, dtype=torch.bfloat16)
    bias, offs = ints(g, (N,), -9, 9, torch.float32), offsets_of(counts)
    D = torch.empty(193, N, device=DEV)
    tge.QuantPlan(193, N, K, 64, 4, stride_bias=0, ab="bf16", cd="f32", epilogue="bias", algo=algo, tile=tile).run(
        A.to(DEV), Q.to(DEV), scales.to(DEV), None, None, D, torch.from_numpy(offs).to(DEV), bias.to(DEV))
    W = dequantised(Q, scales, None, 64)
    for e in range(4):
        lo, hi = offs[e], offs[e + 1]
        assert torch.equal(D[lo:hi].cpu().double(), A[lo:hi].double() @ W[e].t() + bias.double())


@pytest.mark.parametrize("ab,cd", [("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("algo,tile", [("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128), ("staged", 64),
                                       ("skinny", 0), ("skinny", 64), ("general", 128), ("general", 64)])
def test_gate_with_nan_and_infinities(algo, tile, ab, cd):
    # NaN in C closes the gate like any value that is not above 0 (so do -0 and -inf), and a closed
    # gate gives 0 whatever the product is
    g = np.random.default_rng(5)
    counts, N, K = [40, 0, 300, 3], 264, 64
    T = sum(counts)
    A, B = ints(g, (T, K), -3, 3, TORCH_DT[ab]), ints(g, (4, N, K), -3, 3, TORCH_DT[ab])
    A[7], A[200, 3], A[342] = NAN, INF, -INF
    C = ints(g, (T, N), -2, 2, TORCH_DT[cd])
    C[torch.from_numpy(g.random((T, N)) < 0.2)] = NAN
    C[5], C[6], C[7, ::2], C[8] = INF, -INF, -0.0, -0.0
    offs = offsets_of(counts)
    D = torch.full((T, N), SENTINEL, dtype=TORCH_DT[cd], device=DEV)
    tge.GroupedPlan(T, N, K, 4, "T", ab=ab, cd=cd, epilogue="gate", algo=algo, tile=tile).run(
        A.to(DEV), B.to(DEV), C.to(DEV), D, torch.from_numpy(offs).to(DEV))
    want = torch.zeros(T, N, dtype=torch.float64)
    for e in range(4):
        for r in range(offs[e], offs[e + 1]):
            want[r] = torch.where(C[r] > 0, (A[r].double()[None] * B[e].double()).sum(1), 0.0)
    want, got = rounded(want, TORCH_DT[cd]), D.cpu()
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())
