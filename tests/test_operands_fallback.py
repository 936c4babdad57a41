"""The plans that check a run's tensors in one call of the module _operands work where it is not built, or was
built for another torch: the checks one by one take its place."""
import sys

import pytest
import torch

import tiled_gemm_epilogues_amd as tge


@pytest.fixture(params=["missing", "other torch"])
def without(request, monkeypatch):
    if request.param == "missing":
        monkeypatch.delattr(tge, "_operands", raising=False)
        monkeypatch.delitem(sys.modules, tge.__name__ + "._operands", raising=False)
        monkeypatch.setattr(tge, "__path__", [])
        with pytest.raises(ImportError):
            from tiled_gemm_epilogues_amd import _operands
    else:
        from tiled_gemm_epilogues_amd import _operands
        assert _operands.torch_version == str(torch.__version__)
        monkeypatch.setattr(_operands, "torch_version", "0.0")


def plans():
    return [(tge.LayerPlan(4, 8, 16), "A"), (tge.NormPlan(4, 8, "f32"), "X"), (tge.RoutePlan(4, 8, 2), "logits")]


def test_plans_without_the_module(without):
    with pytest.warns(RuntimeWarning, match="_operands"):
        made = plans()
    for p, first in made:
        n = len(p._RUN)
        assert tuple(p._pointers(0, *range(n))) == tuple(range(n))
        assert tuple(p._grad_pointers(0, *[None] * len(p._GRAD))) == (None,) * len(p._GRAD)
        with pytest.raises(ValueError, match=f"{first} must be a device tensor"):
            p._pointers(0, torch.zeros(4, 16), *[None] * (n - 1))


def test_plans_with_the_module(recwarn):
    from tiled_gemm_epilogues_amd import _operands
    for p, _ in plans():
        assert isinstance(p._run_fits, _operands.Operands) and isinstance(p._grad_fits, _operands.Operands)
    assert not [w for w in recwarn if "_operands" in str(w.message)]


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore:.*_operands")
def test_runs_without_the_module(without):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    p = tge.NormPlan(40, 96, "f32")
    g = torch.Generator().manual_seed(1)
    X, dY, w = (torch.randn(*s, generator=g).to("cuda:0") for s in ((40, 96), (40, 96), (96,)))
    new = lambda *s: torch.full(s, float("nan"), device="cuda:0")
    got = [new(40, 96), new(40), new(40), new(40, 96), new(96), new(96)]
    p.run(X, w, None, *got[:3])
    p.run_grad(dY, X, w, *got[1:])
    with pytest.raises(TypeError, match="weight"):
        p.run(X, w.double(), None, *got[:3])
    x = X.double().requires_grad_()
    ww = w.double().requires_grad_()
    y = torch.nn.functional.layer_norm(x, (96,), ww)
    y.backward(dY.double())
    # 96 values of size 1 to 3, some tens of roundings
    for a, b in zip((got[0], got[3], got[4], got[5]), (y, x.grad, ww.grad, dY.double().sum(0))):
        assert (a.double() - b).abs().max() < 2e-5
