"""Rows without a logit above minus infinity, NaN among them or nothing else: they are left out like masked
ones, whatever else is in them, in every shape of lanes and for few and many rows."""
import pytest
import torch

from grouped_helpers import TORCH_DT
from test_route_gpu import Run, check, logits_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gradient(r, dw, dloss):
    out = torch.full_like(r.logits, 7.0)
    r.plan.run_grad(r.logits, r.index, dw, r.slope, torch.full((1,), dloss, device=DEV), out, r.mask)
    return out


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E,k,T", [(1, 1, 20), (5, 2, 50), (16, 4, 40000), (24, 4, 30), (24, 4, 600), (60, 6, 40000), (128, 8, 33),
                                   (129, 12, 700), (256, 8, 20000), (500, 16, 90), (1000, 3, 200)])
def test_rows_of_nan_and_minus_infinity(E, k, T, type, normalize):
    x = logits_of(E + T, T, E, type)
    out = [0, 3, 4, T // 2, T - 2, T - 1]
    x[0], x[3], x[4], x[T // 2], x[T - 2], x[T - 1] = NAN, -INF, NAN, -INF, -INF, NAN
    x[T // 2, E // 2] = NAN                                 # one NaN beside minus infinities
    x[T - 2, 0] = x[T - 2, E - 1] = NAN
    r, index, _, used, _ = check(x, k, type, normalize)
    assert not used[out].any() and (index[out] == -1).all() and (r.weight[out] == 0).all() and int(used.sum()) == T - 6
    # what a mask of these rows gives, bit for bit
    mask = torch.ones(T, dtype=torch.uint8)
    mask[out] = 0
    m = Run(x, k, type, normalize, mask)
    for a, b in zip(r.outputs() + [r.slope, r.loss], m.outputs() + [m.slope, m.loss]):
        assert torch.equal(a, b)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).to(DEV)
    for dloss in (0.5, NAN, INF):
        got, want = gradient(r, dw, dloss), gradient(m, dw, dloss)
        assert (got[out] == 0).all()
        assert torch.equal(got.view(torch.int16 if TORCH_DT[type].itemsize == 2 else torch.int32),
                           want.view(torch.int16 if TORCH_DT[type].itemsize == 2 else torch.int32))
        if dloss == 0.5:
            assert got.isfinite().all()


def test_nan_beside_a_logit_is_not_left_out():
    x = logits_of(3, 70, 20, "f32")
    x[1], x[1, 4], x[1, 6] = -INF, NAN, 1.0
    r = Run(x, 3, "f32", False)
    assert r.index[1].tolist() == [6, -1, -1] and r.weight[1, 0].isnan() and r.loss.isnan().all()
    dw = torch.zeros(70, 3, device=DEV)
    assert gradient(r, dw, 1.0)[1].isnan().any()
