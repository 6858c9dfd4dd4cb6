"""Layer norm of features without positions."""
import pytest
import torch

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


@pytest.mark.parametrize("shape", [(2, 16, 0), (3, 16, 0, 7), (2, 16, 5, 0), (0, 16, 0)])
def test_empty_planes(shape):
    x = torch.empty(shape, device="cuda", dtype=torch.float16)
    w = torch.ones(16, device="cuda")
    y, mean, rstd = fc.layer_norm(x, w, w, axis=1, return_stats=True)
    assert y.shape == shape and mean.shape == rstd.shape == shape[:1] + shape[2:]
    dx, dw, db = fc.layer_norm_backward(x, x, mean, rstd, w, w, axis=1)
    assert dx.shape == shape
    assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0
