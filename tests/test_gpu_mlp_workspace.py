"""Both passes of the gated block over a workspace and a `saved` that hold NaN, at sizes that end inside
their units: nothing that a call did not write itself is read into a result."""
import pytest
import torch

import block_ref as B
import ops_ref as R
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops
from test_gpu_mlp import NAMES, case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    _ops._start()
    yield
    _ops.check_device()


def nan(nbytes):
    return torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("route", ["auto", "simple"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,f,o", [(7, 33, 61, 19), (45, 72, 130, 56), (70, 37, 131, 61),
                                     (333, 264, 517, 203)])
@pytest.mark.parametrize("kept", [True, False])
def test_nothing_left_over_is_read(n, c, f, o, dtype, route, kept):
    x, wg, wu, wd, b, dy = case(700, n, c, f, o, R.TYPES[dtype])
    dev = [t.contiguous().cuda() for t in (x, wg, wu, wd, *b)]
    p = fc.MlpPlan(_ops._code(x.dtype), n, c, f, o, x_stride=c, y_stride=o, gate_stride=c,
                   up_stride=c, down_stride=f, dy_stride=o, dx_stride=c, has_b_gate=True,
                   has_b_up=True, has_b_down=True, training=True, route=route)
    stream = torch.cuda.current_stream().cuda_stream
    at = [t.data_ptr() for t in dev]
    new = lambda *s: torch.full(s, float("nan"), dtype=x.dtype, device="cuda")  # noqa: E731
    y, saved, ws = new(n, o), nan(p.saved_bytes), nan(p.forward_workspace)
    p.forward_ptrs(*at, y.data_ptr(), saved.data_ptr() if kept else None, ws.data_ptr(), ws.numel(),
                   stream)
    outs = [new(n, c), new(f, c), new(f, c), new(o, f), new(f), new(f), new(o)]
    ws2 = nan(p.backward_workspace)
    grad = dy.cuda()
    p.backward_ptrs(grad.data_ptr(), *at[:6], saved.data_ptr() if kept else None,
                    *(t.data_ptr() for t in outs), ws2.data_ptr(), ws2.numel(), stream)
    torch.cuda.synchronize()
    got = {"y": y, **dict(zip(NAMES, outs))}
    for name, (val, tol) in B.gated_mlp(x, wg, wu, wd, *b, dy=dy).items():
        R.check(got[name], val, tol, name)
