"""Head norms of very large and very small heads: right as long as the squares' sum is an f32, zeros
past it."""
import pytest
import torch

import block_ref as B
import ops_ref as R
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    yield
    _ops.check_device()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale,eps", [(1e17, 1e-6), (1e17, 1e30), (1e-14, 1e-30), (1e-9, 1e-6),
                                       (1.0, 1e-30), (1e6, 1e-38)])
@pytest.mark.parametrize("d", [64, 33])
def test_sizes_of_heads(dtype, scale, eps, d):
    T = R.TYPES[dtype]
    q, dq, w = R.normal(1, (1, 9, 3, d), T, scale), R.normal(2, (1, 9, 3, d), T), \
        R.normal(3, (d,), T, 0.2, 1.0)
    pos = torch.arange(9, dtype=torch.int32)[:, None]
    freq, sections = fc.rope_frequencies((d // 2,), device="cpu"), (d // 2,)
    how = dict(weight=w.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(), eps=eps)
    eps = torch.tensor(eps, dtype=torch.float32).double()  # as the call holds it
    R.check(fc.norm_rope(q.cuda(), **how), *B.norm_rope(q, w, pos, freq, sections, "half", eps), "y")
    dx, _, dw, _ = fc.norm_rope_backward(dq.cuda(), q.cuda(), **how)
    ref = B.norm_rope_backward(dq, q, w, pos, freq, sections, "half", eps)
    R.check(dx, *ref["dx"], "dx")
    R.check(dw, *ref["dw"], "dw")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_heads_whose_squares_no_f32_holds(dtype):
    q = R.normal(4, (1, 5, 2, 64), R.TYPES[dtype])
    q[0, 2, 1] *= 1e25
    y = fc.norm_rope(q.cuda()).cpu()
    assert (y[0, 2, 1] == 0).all()
    y[0, 2, 1], q[0, 2, 1] = 0, 0
    R.check(y, *B.norm_rope(q, None, None, None, None, "half", 1e-6), "y")
