"""Products with 4-bit weights on the GPU, against the definition in 64 bits.  Small integer
activations and biases with scales that are powers of two make every fp32 step exact, so the
outputs must equal the rounded reference bit for bit; one test uses random values, with a bound
counted from the roundings."""
import numpy as np
import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import SENTINEL, TORCH_DT, ints, offsets_of, rounded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dequantised(Q, scales, zeros, block):
    """The weights in 64 bits, experts x N x K."""
    E, N, half = Q.shape
    q = torch.stack([Q & 15, Q >> 4], dim=-1).reshape(E, N, 2 * half).double()
    near = torch.arange(2 * half) // block
    z = zeros.double()[..., near] if zeros is not None else 8.0
    return (q - z) * scales.double()[..., near]


def reference(A, W, C, D0, offs, bias, alpha, beta, epilogue):
    D = D0.double().clone()
    for e, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        if lo == hi:
            continue
        d = alpha * (A[lo:hi].double() @ W[e].t())
        if beta:
            d = d + beta * C[lo:hi].double()
        if "bias" in epilogue:
            d = d + bias[e].double()
        if "relu" in epilogue:
            d = torch.clamp(d, min=0)
        D[lo:hi] = d
    return D


def wide(x, ld, fill):
    out = torch.full((*x.shape[:-1], ld), fill, dtype=x.dtype)
    out[..., :x.shape[-1]] = x
    return out


def quant_case(counts, N, K, block, zeros=False, ab="f16", cd="f16", epilogue="none", alpha=1.0,
               beta=0.0, start=0, behind=0, dense=False, pads=0, offset=0, algo="auto", tile=0,
               kernel=None, in_place=False, seed=0):
    g = np.random.default_rng(seed)
    offs = offsets_of(counts, start)
    T, E, nb = int(offs[-1]) + behind, len(counts), K // block
    tab, tcd = TORCH_DT[ab], TORCH_DT[cd]
    A = ints(g, (T, K), -3, 3, tab)
    used = torch.zeros(T, dtype=torch.bool)
    used[offs[0]:offs[-1]] = True
    A[~used] = float("nan")
    Q = torch.from_numpy(g.integers(0, 256, (E, N, K // 2)).astype(np.uint8))
    scales = torch.from_numpy(2.0 ** g.integers(-1, 2, (E, N, nb))).to(tab)
    z = torch.from_numpy(g.integers(0, 16, (E, N, nb)).astype(np.uint8)) if zeros else None
    bias = ints(g, (E, N), -9, 9, torch.float32)
    C = ints(g, (T, N), -9, 9, tcd)
    lda, ldq, lds, ldc = max(K, 1) + 3 * pads, K // 2 + pads, nb + pads, N + pads
    D0 = wide(C, ldc, float("nan")) if in_place else torch.full((T, ldc), SENTINEL, dtype=tcd)
    p = tge.QuantPlan(T, N, K, block, E, zeros, lda, ldq, lds, ldc, ab=ab, cd=cd, epilogue=epilogue,
                      algo=algo, tile=tile)
    if kernel:
        assert kernel in p.describe(), p.describe()

    def dev(x):      # `offset` elements off the allocation's alignment
        flat = torch.cat([torch.zeros(offset, dtype=x.dtype), x.reshape(-1)]).to(DEV)
        return flat[offset:]

    D = dev(D0)
    dC = (D if in_place else dev(wide(C, ldc, float("nan")))) if beta else None
    p.run(dev(wide(A, lda, float("nan"))), dev(wide(Q, ldq, 255)), dev(wide(scales, lds, float("nan"))),
          dev(wide(z, lds, 255)) if zeros else None, dC, D,
          None if dense else torch.from_numpy(offs).to(DEV), dev(bias) if "bias" in epilogue else None,
          alpha, beta)
    torch.cuda.synchronize()
    want = reference(A, dequantised(Q, scales, z, block), C, D0[:, :N], offs, bias, alpha, beta, epilogue)
    expect = D0.clone()
    expect[:, :N] = rounded(want, tcd)
    got = D.cpu().reshape(T, ldc)
    bad = ~((got == expect) | (got.isnan() & expect.isnan()))
    assert not bad.any(), f"{p.describe()}: {int(bad.sum())} differ, first {bad.nonzero()[0].tolist()}"


KERNELS = [("skinny", 16), ("skinny", 64), ("fast", 128)]


@pytest.mark.parametrize("block", [32, 64, 128, 256])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("ab", ["f16", "bf16"])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_every_kernel_block_and_type(algo, tile, ab, zeros, block):
    name = "quant_tile" if algo == "fast" else "quant_rows"
    quant_case([77], 150, 768, block, zeros, ab, "f32", "bias", dense=True, algo=algo, tile=tile,
               kernel=name, seed=block)
    quant_case([5, 0, 130, 1], 72, 256, block, zeros, ab, ab, "bias_relu", start=2, behind=3,
               algo=algo, tile=tile, seed=block + 1)


@pytest.mark.parametrize("block,K", [(32, 32), (32, 96), (32, 160), (64, 64), (64, 192), (128, 128),
                                     (384, 384), (32, 0), (32, 4128)])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_short_and_partial_chunks(algo, tile, block, K):
    for ab in ("f16", "bf16"):
        quant_case([19], 40, K, block, True, ab, "f32", "bias", dense=True, algo=algo, tile=tile, seed=K)


@pytest.mark.parametrize("rows,N", [(1, 1), (1, 17), (3, 16), (16, 15), (17, 129), (64, 31), (65, 128),
                                    (129, 130), (300, 5)])
def test_odd_sizes(rows, N):
    for zeros in (False, True):
        quant_case([rows], N, 640, 128, zeros, "bf16", "f32", dense=True, seed=rows)
        quant_case([rows], N, 640, 64, zeros, "f16", "f16", dense=True, seed=rows + 1)


@pytest.mark.parametrize("algo,tile", KERNELS)
def test_epilogues_scalars_in_place(algo, tile):
    for epilogue in ("none", "relu", "bias", "bias_relu"):
        quant_case([40, 30], 24, 256, 64, False, "f16", "f32", epilogue, alpha=-2.0, beta=1.0, algo=algo,
                   tile=tile, seed=3)
    quant_case([40, 30], 24, 256, 64, True, "bf16", "bf16", "relu", beta=2.0, in_place=True, algo=algo,
               tile=tile, seed=4)


@pytest.mark.parametrize("algo,tile", KERNELS)
def test_strides_and_unaligned_pointers(algo, tile):
    quant_case([33, 0, 20], 24, 256, 64, True, "f16", "f32", "bias", beta=1.0, pads=1, offset=1,
               algo=algo, tile=tile, seed=5)
    quant_case([33, 0, 20], 24, 256, 128, True, "bf16", "bf16", "bias", beta=1.0, pads=5, offset=3,
               algo=algo, tile=tile, seed=6)


@pytest.mark.parametrize("algo,tile", KERNELS)
def test_rows_far_apart(algo, tile):
    # rows of A 2^24 bytes and more apart: 128 of them span 2^31
    g = np.random.default_rng(8)
    rows, N, K, block, lda = 40, 40, 320, 64, (1 << 23) + 8
    A = ints(g, (rows, K), -3, 3, torch.float16)
    Q = torch.from_numpy(g.integers(0, 256, (1, N, K // 2)).astype(np.uint8))
    scales = torch.from_numpy(2.0 ** g.integers(-1, 2, (1, N, K // block))).to(torch.float16)
    dA = torch.empty(rows, lda, dtype=torch.float16, device=DEV)
    dA[:, :K] = A.to(DEV)
    D = torch.empty(rows, N, dtype=torch.float32, device=DEV)
    tge.QuantPlan(rows, N, K, block, 1, False, lda, ab="f16", cd="f32", algo=algo, tile=tile).run(
        dA, Q.to(DEV), scales.to(DEV), None, None, D)
    want = A.double() @ dequantised(Q, scales, None, block)[0].t()
    assert (D.cpu().double() == want).all()


@pytest.mark.parametrize("counts,start,behind", [([0], 0, 2), ([1] * 130, 1, 0), ([0, 0, 9], 0, 0),
                                                ([200], 3, 3), ([16, 32, 64, 128], 0, 0)])
@pytest.mark.parametrize("algo,tile", [("auto", 0), *KERNELS])
def test_ranges(counts, start, behind, algo, tile):
    quant_case(counts, 20, 128, 64, True, start=start, behind=behind, algo=algo, tile=tile, seed=7)


@pytest.mark.parametrize("algo,tile", KERNELS)
@pytest.mark.parametrize("ab,cd", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_random_values(algo, tile, ab, cd):
    # Bound: |A| (15 + 24)-weighted: a block's terms A * (16 + q) and (16 + z) * sum A are at most
    # 31 |A| each; each of the at most K + K / block + 4 fp32 additions and scalings is off by one
    # step (2^-23, twice a rounding to nearest) of a partial result no larger than the sum of the
    # terms' magnitudes, and the output rounding by half a step of its type.
    g = torch.Generator().manual_seed(8)
    rows, N, K, block = 70, 72, 1024, 64
    A = torch.randn(rows, K, generator=g).to(TORCH_DT[ab])
    Q = torch.randint(0, 256, (1, N, K // 2), generator=g, dtype=torch.uint8)
    scales = ((torch.rand(1, N, K // block, generator=g) + 0.5) / 64).to(TORCH_DT[ab])
    zeros = torch.randint(0, 16, (1, N, K // block), generator=g, dtype=torch.uint8)
    D = torch.empty(rows, N, dtype=TORCH_DT[cd], device=DEV)
    tge.QuantPlan(rows, N, K, block, zeros=True, ab=ab, cd=cd, algo=algo, tile=tile).run(
        A.to(DEV), Q.to(DEV), scales.to(DEV), zeros.to(DEV), None, D)
    ref = A.double() @ dequantised(Q, scales, zeros, block)[0].t()
    near = torch.arange(K) // block
    mag = A.abs().double() @ (62 * scales[0].double()[:, near]).t()
    acc = (K + K // block + 4) * 2.0 ** -23 * mag
    half = 0.0 if cd == "f32" else torch.finfo(TORCH_DT[cd]).eps / 2
    tol = acc + half * (ref.abs() + acc) + (2.0 ** -25 if cd == "f16" else 0.0)
    assert ((D.cpu().double() - ref).abs() <= tol).all()


def test_beyond_32_bit_offsets():
    # the last expert's codes start beyond 2^32 bytes, the used rows of A too
    E, N, K, T = 1030, 2048, 4096, 600_000
    g = np.random.default_rng(9)
    Q = torch.zeros(E, N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.ones(E, N, K // 128, dtype=torch.float16, device=DEV)
    A = torch.empty(T, K, dtype=torch.float16, device=DEV)
    q = torch.from_numpy(g.integers(0, 256, (N, K // 2)).astype(np.uint8))
    Q[E - 1] = q.to(DEV)
    tail = ints(g, (90, K), -1, 1, torch.float16)
    A[T - 90:] = tail.to(DEV)
    offs = torch.tensor([T - 90] * E + [T], dtype=torch.int32, device=DEV)
    D = torch.empty(T, N, dtype=torch.float32, device=DEV)
    want = tail.double() @ dequantised(q[None], torch.ones(1, N, K // 128), None, 128)[0].t()
    for algo, tile in KERNELS:
        D[T - 91:] = SENTINEL
        tge.QuantPlan(T, N, K, 128, E, cd="f32", algo=algo, tile=tile).run(A, Q, scales, None, None, D, offs)
        assert (D[T - 91] == SENTINEL).all()
        assert torch.equal(D[T - 90:].cpu(), want.float()), f"{algo} {tile}"
