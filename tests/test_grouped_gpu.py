"""Products grouped by expert on the GPU (rows and gradient plans), against the definition in 64
bits.  The inputs are small integers: every product and fp32 partial sum is exact, so the outputs
must equal the rounded reference bit for bit whatever the kernel and its order of summation.  One
test per mode uses random values, with a bound counted from the roundings."""
import numpy as np
import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import (SENTINEL, TORCH_DT, grad_reference, ints, offsets_of, rounded,
                             rows_reference)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def padded(x, ld):
    """x with rows of ld elements (the padding holds a value that must never be used)."""
    out = torch.full((*x.shape[:-1], ld), float("nan"), dtype=x.dtype)
    out[..., :x.shape[-1]] = x
    return out


def same(got, want, what):
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), f"{what}: {int(bad.sum())} differ, first {bad.nonzero()[0].tolist()}"


def rows_case(counts, N, K, op_b="N", ab="f16", cd="f16", epilogue="none", alpha=1.0, beta=0.0,
              start=0, behind=0, lda=None, ldb=None, ldc=None, algo="auto", tile=0, kernel=None,
              share_b=False, in_place=False, seed=0):
    g = np.random.default_rng(seed)
    offs = offsets_of(counts, start)
    T, E = int(offs[-1]) + behind, len(counts)
    tab, tcd = TORCH_DT[ab], TORCH_DT[cd]
    lda, ldc = lda or max(K, 1), ldc or N
    ldb = ldb or (N if op_b == "N" else max(K, 1))
    A = ints(g, (T, K), -3, 3, tab)
    used = torch.zeros(T, dtype=torch.bool)
    used[offs[0]:offs[-1]] = True
    A[~used] = float("nan")                 # rows of nobody: never read into a result
    B = ints(g, (1 if share_b else E, *((K, N) if op_b == "N" else (N, K))), -3, 3, tab)
    bias = ints(g, (E, N), -9, 9, torch.float32)
    C = ints(g, (T, N), -9, 9, tcd)
    D0 = padded(C, ldc) if in_place else torch.full((T, ldc), SENTINEL, dtype=tcd)
    needs_c = beta != 0 or epilogue == "gate"
    p = tge.GroupedPlan(T, N, K, E, op_b, lda, ldb, ldc, stride_b=0 if share_b else None, ab=ab,
                        cd=cd, epilogue=epilogue, algo=algo, tile=tile)
    if kernel:
        assert kernel in p.describe(), p.describe()
    D = D0.to(DEV)
    dC = (D if in_place else padded(C, ldc).to(DEV)) if needs_c else None
    p.run(padded(A, lda).to(DEV), padded(B, ldb).to(DEV), dC, D, torch.from_numpy(offs).to(DEV),
          bias.to(DEV) if "bias" in epilogue else None, alpha, beta)
    torch.cuda.synchronize()
    want = rows_reference(A, B, C, D0[:, :N], offs, op_b, bias, alpha, beta, epilogue)
    out = D.cpu()
    same(out[:, :N], rounded(want, tcd), f"{p.describe()} {counts}")
    same(out[:, N:], D0[:, N:], "padding of D")


RAGGED = [5, 0, 130, 1, 64, 0, 0, 300, 17]
KERNELS = [("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128), ("staged", 64), ("skinny", 0), ("skinny", 64),
           ("general", 128), ("general", 64)]
NAMES = {"fast": "gemm_fast", "staged": "_rs", "skinny": "gemm_rows16",
         "general": "gemm_mfma"}


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_rows_every_kernel(algo, tile, op_b):
    name = NAMES[algo]
    rows_case(RAGGED, 200, 160, op_b, "f16", "f16", "bias_relu", alpha=2.0, beta=-1.0, start=3,
              behind=11, algo=algo, tile=tile, kernel=name, seed=tile)


@pytest.mark.parametrize("ab,cd", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                   ("f32", "f32")])
@pytest.mark.parametrize("algo,tile", [("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128), ("staged", 64),
                                       ("skinny", 0), ("skinny", 64), ("general", 64)])
def test_rows_types(ab, cd, algo, tile):
    rows_case([40, 3, 0, 257], 136, 192, "T", ab, cd, "gate", start=1, behind=2, algo=algo,
              tile=tile, seed=1)


@pytest.mark.parametrize("epilogue", ["none", "relu", "bias", "bias_relu", "gate"])
@pytest.mark.parametrize("algo,tile", [("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128), ("staged", 64),
                                       ("skinny", 64), ("general", 128)])
def test_rows_epilogues(epilogue, algo, tile):
    beta = 0.0 if epilogue == "gate" else 2.0
    rows_case([33, 200, 0, 90], 264, 128, "N", "bf16", "f32", epilogue, alpha=-1.0, beta=beta,
              algo=algo, tile=tile, seed=2)
    rows_case([33, 200, 0, 90], 264, 128, "N", "f16", "f16", epilogue, beta=beta, algo=algo,
              tile=tile, in_place=True, seed=3)


@pytest.mark.parametrize("counts,start,behind", [
    ([1], 0, 0), ([0], 0, 1), ([0, 0, 0], 2, 0), ([0, 1], 0, 0), ([1] * 130, 0, 0),
    ([0] * 64 + [1], 0, 5), ([3, 0] * 100, 1, 1), ([700], 0, 0), ([0] * 299 + [129], 7, 0),
    ([2] * 64, 0, 0), ([128, 256, 64], 0, 0)])
@pytest.mark.parametrize("algo,tile", [("auto", 0), ("fast", 128), ("fast", 64), ("staged", 128), ("staged", 64), ("skinny", 0), ("skinny", 64),
                                       ("general", 64)])
def test_rows_ranges(counts, start, behind, algo, tile):
    rows_case(counts, 72, 64, "T", start=start, behind=behind, algo=algo, tile=tile, seed=4)


@pytest.mark.parametrize("N,K", [(1, 1), (7, 3), (8, 64), (77, 65), (129, 1001), (1000, 31),
                                 (64, 63), (300, 0), (8, 8192)])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_rows_odd_sizes(N, K, op_b):
    for ab, cd in (("f16", "f16"), ("f32", "f32")):
        rows_case([5, 0, 40, 1, 150], N, K, op_b, ab, cd, "bias", start=1, behind=1, seed=5)


@pytest.mark.parametrize("algo,tile", [("staged", 128), ("staged", 64), ("skinny", 0), ("skinny", 64), ("general", 64)])
@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("N,K", [(8, 8), (9, 15), (63, 63), (65, 64), (71, 65), (127, 129), (129, 200),
                                 (64, 128), (72, 513), (1001, 1001)])
def test_rows_edges_of_every_kernel(N, K, op_b, algo, tile):
    # nothing behind the last row or expert: a load past an operand's end would leave its memory
    rows_case([5, 0, 40, 1, 15], N, K, op_b, "bf16", "f32", "bias", algo=algo, tile=tile, seed=N)


def test_rows_strides_and_shared_weights():
    rows_case([50, 20, 300], 96, 128, "N", lda=136, ldb=104, ldc=120, seed=6)
    rows_case([50, 20, 300], 96, 128, "T", lda=131, ldb=129, ldc=97, seed=7)
    rows_case([50, 20, 300], 96, 128, "T", share_b=True, algo="fast", seed=8)


def test_rows_unaligned_pointers():
    # the plan's fast kernel needs 16-byte aligned A and B: the general one runs instead
    g = np.random.default_rng(9)
    offs = offsets_of([100, 60])
    A, B = ints(g, (160, 128), -3, 3, torch.float16), ints(g, (2, 128, 64), -3, 3, torch.float16)
    dA, dB = (torch.cat([torch.zeros(1, dtype=torch.float16), x.reshape(-1)]).to(DEV)[1:] for x in (A, B))
    D = torch.full((160 * 64 + 1,), SENTINEL, dtype=torch.float16, device=DEV)
    p = tge.GroupedPlan(160, 64, 128, 2, algo="fast")
    assert "gemm_fast" in p.describe()
    p.run(dA, dB, None, D[1:], torch.from_numpy(offs).to(DEV))
    want = rows_reference(A, B, None, torch.zeros(160, 64), offs, "N", None, 1.0, 0.0, "none")
    same(D[1:].cpu().reshape(160, 64), rounded(want, torch.float16), "unaligned")
    assert D[0].item() == SENTINEL


@pytest.mark.parametrize("algo,tile", [("fast", 128), ("fast", 64), ("staged", 64), ("skinny", 0), ("general", 64)])
def test_rows_unordered_offsets_stay_inside(algo, tile):
    # undefined results, but nothing outside D's rows is written
    T, N, K = 100, 64, 64
    A = torch.ones(T, K, dtype=torch.float16, device=DEV)
    B = torch.ones(4, K, N, dtype=torch.float16, device=DEV)
    buf = torch.full((T + 400, N), SENTINEL, dtype=torch.float16, device=DEV)
    offs = torch.tensor([0, 250, -7, 60, 2000000000], dtype=torch.int32, device=DEV)
    tge.GroupedPlan(T, N, K, 4, algo=algo, tile=tile).run(A, B, None, buf[200:200 + T], offs)
    out = buf.cpu()
    assert (out[:200] == SENTINEL).all() and (out[200 + T:] == SENTINEL).all()


def test_rows_beyond_32_bit_offsets():
    # A and D pass 2^32 bytes: the ranges lie at the far end
    T, N, K = 600_000, 1024, 4096
    g = np.random.default_rng(10)
    A = torch.empty(T, K, dtype=torch.float16, device=DEV)
    D = torch.empty(T, N, dtype=torch.float32, device=DEV)
    tail = 700
    A[T - tail:] = ints(g, (tail, K), -1, 1, torch.float16).to(DEV)
    B = ints(g, (3, N, K), -1, 1, torch.float16)
    offs = offsets_of([100, 300, 290], T - tail)
    for algo, tile in (("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128), ("staged", 64), ("skinny", 64), ("skinny", 16),
                       ("general", 128)):
        D[T - tail:] = SENTINEL
        tge.GroupedPlan(T, N, K, 3, "T", cd="f32", algo=algo, tile=tile).run(
            A, B.to(DEV), None, D, torch.from_numpy(offs).to(DEV))
        want = rows_reference(A[T - tail:].cpu(), B, None, torch.full((tail, N), SENTINEL),
                              offs - (T - tail), "T", None, 1.0, 0.0, "none")
        same(D[T - tail:].cpu(), rounded(want, torch.float32), f"{algo} {tile}")


def grad_case(counts, M, N, ab="f16", cd="f32", alpha=1.0, beta=0.0, start=0, behind=0, lda=None,
              ldb=None, ldc=None, extra=0, algo="auto", tile=0, kernel=None, bias=True,
              in_place=False, seed=0):
    g = np.random.default_rng(seed)
    offs = offsets_of(counts, start)
    T, E = int(offs[-1]) + behind, len(counts)
    tab, tcd = TORCH_DT[ab], TORCH_DT[cd]
    lda, ldb, ldc = lda or max(M, 1), ldb or max(N, 1), ldc or max(N, 1)
    A, B = ints(g, (T, M), -3, 3, tab), ints(g, (T, N), -3, 3, tab)
    used = torch.zeros(T, dtype=torch.bool)
    used[offs[0]:offs[-1]] = True
    A[~used] = float("nan")
    B[~used] = float("nan")
    C = ints(g, (E, M, N), -9, 9, tcd)
    stride = M * ldc + extra
    flat = torch.full((E * stride,), SENTINEL, dtype=tcd)
    view = lambda x: torch.as_strided(x, (E, M, N), (stride, ldc, 1))
    cflat = flat.clone()
    view(cflat).copy_(C)
    p = tge.GroupedGradPlan(T, M, N, E, lda, ldb, ldc, stride, ab=ab, cd=cd, algo=algo, tile=tile)
    if kernel:
        assert kernel in p.describe(), p.describe()
    D = (cflat if in_place else flat).to(DEV)
    dC = D if in_place else cflat.to(DEV)
    sums = torch.full((E, N), SENTINEL, device=DEV)
    p.run(padded(A, lda).to(DEV), padded(B, ldb).to(DEV), dC if beta else None, D,
          torch.from_numpy(offs).to(DEV), sums if bias else None, alpha, beta)
    torch.cuda.synchronize()
    want, want_sums = grad_reference(A, B, C, offs, alpha, beta)
    expect = (cflat if in_place else flat).clone()
    view(expect).copy_(rounded(want, tcd))
    same(D.cpu(), expect, p.describe())
    same(sums.cpu(), want_sums.float() if bias else torch.full((E, N), SENTINEL), "bias_grad")


GRAD_KERNELS = [("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128), ("staged", 64), ("general", 128), ("general", 64)]


@pytest.mark.parametrize("ab,cd", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                   ("f32", "f32")])
@pytest.mark.parametrize("algo,tile", GRAD_KERNELS)
def test_grad_every_kernel(algo, tile, ab, cd):
    kernel = NAMES[algo] if ab != "f32" else "gemm_mfma"
    grad_case(RAGGED, 264, 136, ab, cd, start=2, behind=5, algo=algo, tile=tile, kernel=kernel,
              seed=11)


@pytest.mark.parametrize("algo,tile", GRAD_KERNELS)
def test_grad_scalars_and_in_place(algo, tile):
    grad_case([70, 0, 129], 72, 200, alpha=-2.0, beta=1.0, algo=algo, tile=tile, seed=12)
    grad_case([70, 0, 129], 72, 200, "bf16", "bf16", alpha=1.0, beta=1.0, in_place=True, algo=algo,
              tile=tile, seed=13)


@pytest.mark.parametrize("counts,start,behind", [
    ([1], 0, 0), ([0], 0, 3), ([0, 0], 0, 0), ([64], 0, 0), ([63, 64, 65, 128, 127, 129], 0, 1),
    ([1] * 70, 3, 0), ([2000, 0, 1], 0, 0)])
@pytest.mark.parametrize("algo,tile", [("fast", 256), ("fast", 128), ("fast", 64), ("staged", 128), ("staged", 64),
                                       ("general", 64)])
def test_grad_ranges(counts, start, behind, algo, tile):
    grad_case(counts, 64, 72, start=start, behind=behind, algo=algo, tile=tile, seed=14)


@pytest.mark.parametrize("M,N", [(8, 8), (9, 17), (127, 65), (129, 136), (1, 1), (3, 200), (200, 3), (65, 129), (257, 8), (8, 257), (0, 5), (5, 0)])
def test_grad_odd_sizes(M, N):
    for ab in ("f16", "f32"):
        grad_case([5, 0, 90, 1], M, N, ab, "f32", start=1, behind=1, seed=15)
        grad_case([64, 65, 1, 128], M, N, ab, "f32", seed=16)


def test_grad_strides():
    grad_case([90, 10], 64, 80, lda=72, ldb=96, ldc=88, extra=24, seed=16)
    grad_case([90, 10], 64, 80, lda=65, ldb=81, ldc=83, extra=1, bias=False, seed=17)


def test_grad_beyond_32_bit_offsets():
    T, M, N = 600_000, 4096, 128
    g = np.random.default_rng(18)
    A = torch.empty(T, M, dtype=torch.float16, device=DEV)
    B = torch.empty(T, N, dtype=torch.float16, device=DEV)
    tail = 300
    A[T - tail:] = ints(g, (tail, M), -2, 2, torch.float16).to(DEV)
    B[T - tail:] = ints(g, (tail, N), -2, 2, torch.float16).to(DEV)
    offs = offsets_of([100, 0, 190], T - tail)
    want, sums = grad_reference(A[T - tail:].cpu(), B[T - tail:].cpu(), None, offs - (T - tail), 1.0, 0.0)
    for algo, tile in (("fast", 128), ("fast", 256), ("fast", 64), ("staged", 128), ("staged", 64), ("general", 128)):
        D = torch.full((3, M, N), SENTINEL, device=DEV)
        s = torch.full((3, N), SENTINEL, device=DEV)
        tge.GroupedGradPlan(T, M, N, 3, algo=algo, tile=tile).run(
            A, B, None, D, torch.from_numpy(offs).to(DEV), s)
        same(D.cpu(), want.float(), f"{algo} {tile}")
        same(s.cpu(), sums.float(), "bias_grad")


def bound(ref, absref, K, cd):
    """|computed - ref| for fp32 accumulation of K exact products in any order and one rounding to
    cd: each of at most K + 2 additions and scalings is off by one fp32 step at most (2^-23
    relative, twice a rounding to nearest) of a partial result no larger than absref, the sum of
    the terms' magnitudes; the output rounding by half a step of cd (plus a subnormal fp16's)."""
    acc = (K + 2) * 2.0 ** -23 * absref
    half = 0.0 if cd == "f32" else torch.finfo(TORCH_DT[cd]).eps / 2
    return acc + half * (ref.abs() + acc) + (2.0 ** -25 if cd == "f16" else 0.0)


@pytest.mark.parametrize("algo,tile", KERNELS)
@pytest.mark.parametrize("ab,cd", [("f16", "f16"), ("bf16", "f32")])
def test_rows_random_values(algo, tile, ab, cd):
    g = torch.Generator().manual_seed(19)
    counts, N, K = [70, 0, 200, 33], 136, 1024
    offs = offsets_of(counts)
    A = torch.randn(sum(counts), K, generator=g).to(TORCH_DT[ab])
    B = (torch.randn(4, N, K, generator=g) / 32).to(TORCH_DT[ab])
    bias = torch.randn(4, N, generator=g)
    D = torch.empty(sum(counts), N, dtype=TORCH_DT[cd], device=DEV)
    tge.GroupedPlan(sum(counts), N, K, 4, "T", ab=ab, cd=cd, epilogue="bias", algo=algo, tile=tile).run(
        A.to(DEV), B.to(DEV), None, D, torch.from_numpy(offs).to(DEV), bias.to(DEV))
    zero = torch.zeros(sum(counts), N)
    ref = rows_reference(A, B, None, zero, offs, "T", bias, 1.0, 0.0, "bias")
    mag = rows_reference(A.abs(), B.abs(), None, zero, offs, "T", bias.abs(), 1.0, 0.0, "bias")
    assert ((D.cpu().double() - ref).abs() <= bound(ref, mag, K, cd)).all()


@pytest.mark.parametrize("algo,tile", GRAD_KERNELS)
def test_grad_random_values(algo, tile):
    g = torch.Generator().manual_seed(20)
    counts, M, N = [500, 1, 0, 777], 136, 264
    offs = offsets_of(counts)
    A = torch.randn(sum(counts), M, generator=g).bfloat16()
    B = torch.randn(sum(counts), N, generator=g).bfloat16()
    D, s = torch.empty(4, M, N, device=DEV), torch.empty(4, N, device=DEV)
    tge.GroupedGradPlan(sum(counts), M, N, 4, ab="bf16", algo=algo, tile=tile).run(
        A.to(DEV), B.to(DEV), None, D, torch.from_numpy(offs).to(DEV), s)
    ref, sums = grad_reference(A, B, None, offs, 1.0, 0.0)
    mag, smag = grad_reference(A.abs(), B.abs(), None, offs, 1.0, 0.0)
    assert ((D.cpu().double() - ref).abs() <= bound(ref, mag, 777, "f32")).all()
    assert ((s.cpu().double() - sums).abs() <= bound(sums, smag, 777, "f32")).all()
