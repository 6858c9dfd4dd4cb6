"""Host-side tests of the block's calls (no GPU): what the plan of a call is made from."""
import pytest
import torch

from activation_implicit_gemm_gb300 import FconvError, _build, _ops


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


def status(fn, *a):
    try:
        fn(*a)
    except FconvError as e:
        return e.code
    return None


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are none: no GPU may read them")
@pytest.mark.parametrize("dtype,n,shift,odd,warp_level", [
    # 16-bit operands that TMA would read where they are, off 16 bytes: the warp-level kernel
    (1, 100, 2, 0, True), (2, 100, 8, 0, True),
    # rows that TMA does not take are copied whatever their address, and so is all of f32
    (1, 100, 2, 1, False), (1, 100, 0, 1, False), (0, 100, 4, 0, False), (0, 100, 4, 1, False),
    # up to 32 tokens the weights are streamed from any address
    (1, 32, 2, 0, False), (2, 1, 2, 0, False), (1, 33, 2, 0, True),
    (1, 100, 0, 0, False)])
def test_which_calls_reach_the_warp_level_kernel(dtype, n, shift, odd, warp_level):
    """A plan that insists on the tensor-core route refuses just the calls that an automatic one
    gives to the warp-level kernel; the others get as far as a launch, for which there is no GPU."""
    c, f, o = 64, 96, 32
    p = _ops.MlpPlan(dtype, n, c, f, o, x_stride=c + odd, y_stride=o, gate_stride=c + odd,
                     up_stride=c + odd, down_stride=f + odd, dy_stride=o + odd, dx_stride=c,
                     training=True, route="tc")
    at = [(i + 1) << 20 for i in range(16)]
    want = "E_ALIGNMENT" if warp_level else "E_CUDA"
    for i in range(4):  # x, gate, up, down
        ins = [a + (shift if k == i else 0) for k, a in enumerate(at[:4])]
        got = status(p.forward_ptrs, *ins, None, None, None, at[4], None, at[5], 1 << 40, None)
        assert got == want, (i, got)
    for i in range(5):  # dy, x, gate, up, down
        ins = [a + (shift if k == i else 0) for k, a in enumerate(at[:5])]
        got = status(p.backward_ptrs, *ins, None, None, None, *at[5:9], None, None, None, at[9],
                     1 << 40, None)
        # the backward pass has no form of its own for few tokens
        off = dtype and shift and not odd
        assert got == ("E_ALIGNMENT" if off else "E_CUDA"), (i, got)
