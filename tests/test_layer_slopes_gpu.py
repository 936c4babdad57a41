"""The activations of a layer's products and their slopes at finite arguments of any size, in every kernel and
type: the slopes are 0 or 1 far out, whatever the argument's formula grows to."""
import math

import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import TORCH_DT
from layer_helpers import ACTS, A as TANH_A, B as TANH_B, FIT, U, act64, close, phi64, rounding, slope64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")]
KERNELS = [("general", 64), ("general", 128), ("fast", 64), ("fast", 128), ("fast", 256), ("staged", 64),
           ("staged", 128), ("skinny", 64), ("skinny", 16)]
NAMES = {"general": "gemm_mfma", "fast": "gemm_fast", "staged": "_rs", "skinny": "layer_rows"}
SIZES = [3.0, 10.0, 12.0, 14.0, 20.0, 60.0, 75.0, 87.0, 90.0, 100.0, 127.0, 128.0, 1e3, 6e4, 1e9, 1e10, 1e11, 1e13, 2e13, 1e14,
         1e19, 2e19, 1e20, 1e29, 1e30, 1e37, 3e38]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bounds(act, z, dtype):
    """Of |act computed - act64| and |slope computed - slope64| at an exact z, in 64 bits.  Logistic ones: the
    exponent's roundings move e^-|w| by 4 |w| U of it, and s = 1 / (1 + e^-w) by that times 1 - s; eight more roundings.
    The slope's other term has up to three times those of s, on both of its factors.  gelu: the far side's share q has
    (z^2 + 26) U and the fit's error, Phi is q or 1 - q.  An exponential or a logistic below 2^-126 may become 0: with
    it at most z of it (silu 87.4), or z dw/dz in the slope (gelu_tanh 230)."""
    zero = torch.zeros_like(z)
    if act in ("silu", "gelu_tanh"):
        w, dw = (z, torch.ones_like(z)) if act == "silu" else (z * (TANH_A + TANH_B * z * z), TANH_A + 3 * TANH_B * z * z)
        s, t, a = torch.sigmoid(w), torch.sigmoid(-w), w.abs()
        es = s * (4 * a * t + 8) * U
        return z.abs() * es + 88 * 2.0 ** -126, es + (z * dw).abs() * s * t * (12 * a + 24) * U + 232 * 2.0 ** -126
    if act == "gelu":
        p, q = phi64(z), phi64(-z.abs())
        ep = q * ((z * z + 26) * U + FIT[dtype]) + 2 * p * U
        far = (z * torch.exp(-z * z / 2)).abs() / math.sqrt(2 * math.pi)
        return z.abs() * ep + 1e-37, ep + far * (z * z + 6) * U + 1e-37
    return zero, zero


def arguments(dtype):
    """Both signs of the sizes that are finite in `dtype`, and its largest value."""
    top = torch.finfo(dtype).max
    v = torch.tensor([s for s in SIZES if s < top] + [top], dtype=torch.float64).to(dtype)
    return torch.cat([v, -v])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("algo,tile", KERNELS)
@pytest.mark.parametrize("ab,cd", TYPES)
def test_finite_arguments_of_any_size(ab, cd, algo, tile, act):
    tab, tcd = TORCH_DT[ab], TORCH_DT[cd]
    N, K = 72, 64
    # the slope, from a stored argument: a product of 1 times it
    z = arguments(tcd)
    Z = z[:, None].expand(len(z), N).contiguous()
    A, B = torch.zeros(len(z), K, dtype=tab), torch.zeros(N, K, dtype=tab)
    A[:, 0] = B[:, 0] = 1
    plan = tge.LayerPlan(len(z), N, K, ab=ab, cd=cd, act=act, algo=algo, tile=tile)
    assert NAMES[algo] in plan.describe()
    D = torch.full((len(z), N), NAN, dtype=tcd, device=DEV)
    plan.run_grad(A.to(DEV), B.to(DEV), Z.to(DEV), D)
    want = slope64(act, Z.double())
    bound = bounds(act, Z.double(), tcd)[1]
    close(D, want, bound + rounding(want.abs() + bound, tcd) * 1.0001, "slope")
    # the value, of arguments that the product gives
    z = arguments(tab)
    z = z[z.double().abs() <= torch.finfo(tcd).max]
    A = torch.zeros(len(z), K, dtype=tab)
    A[:, 0] = z
    plan = tge.LayerPlan(len(z), N, K, ab=ab, cd=cd, act=act, algo=algo, tile=tile)
    D, P = (torch.full((len(z), N), NAN, dtype=tcd, device=DEV) for _ in range(2))
    plan.run(A.to(DEV), B.to(DEV), None, D, pre=P)
    z = z.double()[:, None].expand(len(z), N)
    assert torch.equal(P.double().cpu(), z)
    want = act64(act, z)
    bound = bounds(act, z, tcd)[0]
    close(D, want, bound + rounding(want.abs() + bound, tcd) * 1.0001, "value")


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("algo,tile", [("general", 64), ("fast", 64), ("staged", 64), ("skinny", 64)])
def test_slope_of_nan_is_nan(algo, tile, act):
    # and at infinity it is the formula's product, 0 times infinity
    rows, N, K = 20, 64, 64
    Z = torch.linspace(-5, 5, rows)[:, None].repeat(1, N)
    Z[3], Z[8, 5], Z[11], Z[12] = NAN, NAN, float("inf"), -float("inf")
    A, B = torch.zeros(rows, K, dtype=torch.bfloat16), torch.zeros(N, K, dtype=torch.bfloat16)
    A[:, 0] = B[:, 0] = 1
    D = torch.zeros(rows, N, device=DEV)
    plan = tge.LayerPlan(rows, N, K, ab="bf16", cd="f32", act=act, algo=algo, tile=tile)
    plan.run_grad(A.to(DEV), B.to(DEV), Z.to(DEV), D)
    assert torch.equal(D.isnan().cpu(), ~Z.isfinite())
