"""Host-side tests of the block's calls (no GPU): what the plan of a call is made from."""
import pytest
import torch

from activation_implicit_gemm_gb300 import _build, _ops


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    _ops._start()


@pytest.mark.parametrize("params", [lambda: [0.75], lambda: (0.75,), lambda: iter([0.75]),
                                    lambda: (v for v in [0.75])])
def test_activation_params_of_any_kind_of_sequence(monkeypatch, params):
    made = []
    real = _ops.MlpPlan

    def plan(*a, **kw):
        made.append(kw["alpha"])
        return real(*a, **kw)

    monkeypatch.setattr(_ops, "MlpPlan", plan)
    monkeypatch.setattr(_ops, "_mlp_plans", {})
    x, w = torch.zeros(5, 8), torch.zeros(8, 8)
    for dx in (None, x):
        _ops._mlp_plan("gated_mlp", x, (w, w, w), (None,) * 3, "QuickGelu", params(), "auto", -1, x,
                       dx)
    assert made == [0.75, 0.75]
    with pytest.raises(ValueError):
        _ops._mlp_plan("gated_mlp", x, (w, w, w), (None,) * 3, "Gelu", params(), "auto", -1, x)
