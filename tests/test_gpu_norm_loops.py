"""Layer norm at sizes where every persistent block takes several rows or tiles: sums of the
parameters' gradients over them, rings that go round, statistics fetched for more than one group
of 32 rows, and parts of which a block adds to what it wrote before. Random data, weight and bias
in f32, against the plain 64-bit form (computed on the GPU for its size)."""
import pytest
import torch

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


SHAPES = [
    # token rows: a warp a row (whole 16-byte units and not), 256 and 512 threads a row
    ("f16", (124001, 96), -1), ("bf16", (122003, 100), -1), ("f32", (123001, 64), -1),
    ("f16", (9001, 512), -1), ("bf16", (7501, 768), -1), ("f16", (7507, 1024), -1),
    ("f16", (15101, 1032), -1), ("f32", (15103, 257), -1), ("f32", (10111, 2056), -1),
    ("bf16", (10103, 2049), -1), ("f16", (5021, 4104), -1), ("f16", (5023, 4099), -1),
    # rows that no block holds
    ("bf16", (1901, 8200), -1), ("f32", (1301, 8193), -1),
    # channels first: staged tiles, many channels, odd 16-bit planes
    ("f16", (5, 24, 70000), 1), ("f32", (5, 24, 35001), 1), ("bf16", (4, 200, 8002), 1),
    ("f32", (4, 200, 4001), 1), ("f16", (3, 256, 12000), 1), ("f16", (3, 300, 12000), 1),
    ("f32", (2, 300, 9001), 1), ("f16", (4, 40, 5431), 1), ("bf16", (2, 300, 9003), 1),
]


@pytest.mark.parametrize("dtype,shape,axis", SHAPES)
def test_forward_and_backward(dtype, shape, axis):
    T, C, eps = R.TYPES[dtype], shape[axis], 1e-5
    g = torch.Generator(device="cuda").manual_seed(7)

    def normal(shape, dtype, scale=1.0, shift=0.0):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (x * scale + shift).to(dtype)

    x, dy = normal(shape, T, 1.5, 0.4), normal(shape, T)
    w, b = normal((C,), torch.float32, 0.3, 1.0), normal((C,), torch.float32, 0.2)
    y, mean, rstd = fc.layer_norm(x, w, b, axis=axis, eps=eps, return_stats=True)
    got = fc.layer_norm_backward(dy, x, mean, rstd, w, b, axis=axis)
    again = fc.layer_norm_backward(dy, x, mean, rstd, w, b, axis=axis)
    ref, m, r, tol = R.layer_norm(x, w, b, axis, eps)

    def check(t, ref, tol, what):
        bad = (t.double() - ref).abs() > tol
        assert not bad.any(), (what, int(bad.sum()), bad.numel())

    check(y, ref, tol, "y")
    e = R.norm_error(x.double().movedim(axis, -1), r)
    check(mean, m, e / r, "mean")
    check(rstd, r, 2 * e * r + 4 * R.E32 * r, "rstd")
    del ref, tol
    want = R.layer_norm_backward(dy, x, w, b, axis, eps)
    for name, t, u in zip(("dx", "dweight", "dbias"), got, again):
        check(t, *want[name], name)
        assert torch.equal(t, u), name
