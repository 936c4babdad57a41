"""Values that products with 4-bit weights meet at the edge of the formula: weights that are exactly
zero, infinities and the largest finite values in A, and zero points over all of a byte.  The kernels
take the sum over a block with the weights code - zero themselves, so each has the result of the
definition, which torch's 64-bit product gives."""
import numpy as np
import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import TORCH_DT, ints
from test_quant_gpu import KERNELS, dequantised

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def product(A, Q, scales, zeros, block, cd, algo, tile):
    """D of one weight matrix, in 64 bits on the CPU."""
    rows, (N, half) = A.shape[0], Q.shape
    ab = {v: k for k, v in TORCH_DT.items()}[A.dtype]
    D = torch.full((rows, N), NAN, dtype=TORCH_DT[cd], device=DEV)
    tge.QuantPlan(rows, N, 2 * half, block, zeros=zeros is not None, ab=ab, cd=cd, algo=algo, tile=tile).run(
        A.to(DEV), Q.to(DEV), scales.to(DEV), None if zeros is None else zeros.to(DEV), None, D)
    return D.cpu().double()


def exact(A, Q, scales, zeros, block):
    W = dequantised(Q[None], scales[None], None if zeros is None else zeros[None], block)[0]
    return torch.stack([(a[None] * W).sum(1) for a in A.double()])


def same(got, want):
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), f"{int(bad.sum())} differ, first {bad.nonzero()[0].tolist()}: {got[bad][0]} for {want[bad][0]}"


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("ab", ["f16", "bf16"])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_codes_at_their_zero_point_give_zero(algo, tile, ab, block):
    # padded or pruned weights: every code is its block's zero point, so that D is 0 whatever A holds
    g = torch.Generator().manual_seed(1)
    rows, N, K = 20, 40, 512
    A = (100 * torch.randn(rows, K, generator=g)).to(TORCH_DT[ab])
    scales = (torch.rand(N, K // block, generator=g) + 0.5).to(TORCH_DT[ab])
    zeros = torch.randint(0, 16, (N, K // block), generator=g, dtype=torch.uint8)
    Q = (zeros * 17).repeat_interleave(block // 2, dim=1)
    assert (product(A, Q, scales, zeros, block, "f32", algo, tile) == 0).all()
    Q = torch.full((N, K // 2), 0x88, dtype=torch.uint8)
    assert (product(A, Q, scales, None, block, "f32", algo, tile) == 0).all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("ab", ["f16", "bf16"])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_infinities_and_nan(algo, tile, ab, zeros):
    # an infinity times a weight is an infinity of the weight's sign, NaN where the weight is 0; rows
    # without one keep their values
    g = np.random.default_rng(2)
    rows, N, K, block = 21, 70, 320, 64
    A = ints(g, (rows, K), -3, 3, TORCH_DT[ab])
    A[1, 5], A[2, 319], A[3, 64], A[4, [10, 300]], A[17, 200] = INF, -INF, NAN, INF, INF
    A[5, 7], A[5, 8] = INF, -INF
    Q = torch.from_numpy(g.integers(0, 256, (N, K // 2)).astype(np.uint8))
    scales = torch.from_numpy(2.0 ** g.integers(-1, 2, (N, K // block))).to(TORCH_DT[ab])
    z = torch.from_numpy(g.integers(0, 16, (N, K // block)).astype(np.uint8)) if zeros else None
    want = exact(A, Q, scales, z, block)
    assert want[1].isinf().any() and want[1].isnan().any() and want[0].isfinite().all()
    same(product(A, Q, scales, z, block, "f32", algo, tile), want)


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_largest_values_stay_finite(algo, tile, block):
    # one value of 2^124 in a row: its products with weights of -8 .. 7 or -15 .. 15 lie below 2^128
    # and are exact in 8 bits
    g = np.random.default_rng(3)
    rows, N, K = 18, 33, 256
    A = torch.zeros(rows, K, dtype=torch.bfloat16)
    A[torch.arange(rows), torch.from_numpy(g.integers(0, K, rows))] = 2.0 ** 124
    Q = torch.from_numpy(g.integers(0, 256, (N, K // 2)).astype(np.uint8))
    scales = torch.ones(N, K // block, dtype=torch.bfloat16)
    z = torch.from_numpy(g.integers(0, 16, (N, K // block)).astype(np.uint8))
    for zeros in (None, z):
        for cd in ("f32", "bf16"):
            same(product(A, Q, scales, zeros, block, cd, algo, tile), exact(A, Q, scales, zeros, block))


@pytest.mark.parametrize("block", [32, 64, 128, 256])
@pytest.mark.parametrize("ab", ["f16", "bf16"])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_zero_points_over_a_byte(algo, tile, ab, block):
    # weights from -255 to 15: sums stay below 2^24 (3 * 255 * 2 * 512), so every step is exact
    g = np.random.default_rng(4)
    rows, N, K = 37, 130, 512
    A = ints(g, (rows, K), -3, 3, TORCH_DT[ab])
    Q = torch.from_numpy(g.integers(0, 256, (N, K // 2)).astype(np.uint8))
    scales = torch.from_numpy(2.0 ** g.integers(-1, 2, (N, K // block))).to(TORCH_DT[ab])
    z = torch.from_numpy(g.integers(0, 256, (N, K // block)).astype(np.uint8))
    z[:4, 0], z[4:8, 0] = 255, 16
    same(product(A, Q, scales, z, block, "f32", algo, tile), exact(A, Q, scales, z, block))


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("ab", ["f16", "bf16"])
@pytest.mark.parametrize("algo,tile", KERNELS)
def test_error_is_that_of_the_weights_themselves(algo, tile, ab, block):
    # Bound: with n nonzero weights in a row, at most n additions inside blocks, n scalings and n
    # additions of parts of the sum round at all (adding 0 does not), each by one fp32 step (2^-23,
    # twice a rounding to nearest) of a partial result no larger than the sum of the terms' magnitudes
    # |A| |code - zero| scale; n = 0 gives 0
    g = torch.Generator().manual_seed(5)
    rows, N, K = 33, 72, 256
    A = torch.randn(rows, K, generator=g).to(TORCH_DT[ab])
    # weights of -1, 0 and 1 with few of them nonzero
    zeros = torch.randint(1, 15, (N, K // block), generator=g, dtype=torch.uint8)
    w = torch.randint(-1, 2, (N, K), generator=g) * (torch.rand(N, K, generator=g) < 0.02)
    q = (zeros.repeat_interleave(block, dim=1).long() + w).to(torch.uint8)
    Q = q[:, 0::2] | (q[:, 1::2] << 4)
    scales = (torch.rand(N, K // block, generator=g) + 0.5).to(TORCH_DT[ab])
    want = exact(A, Q, scales, zeros, block)
    W = dequantised(Q[None], scales[None], zeros[None], block)[0].abs()
    mag = torch.stack([(a[None] * W).sum(1) for a in A.abs().double()])
    n = (w != 0).sum(1).double()
    got = product(A, Q, scales, zeros, block, "f32", algo, tile)
    assert ((got - want).abs() <= 3 * n * 2.0 ** -23 * mag).all()
