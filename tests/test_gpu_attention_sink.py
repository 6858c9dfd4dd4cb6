"""Attention in 16 bits where a few keys outweigh all others but carry no value (sinks): the
output is the sum of the others, whose probabilities are far below the row's largest."""
import math

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


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("above", [16, 18, 20])
@pytest.mark.parametrize("B,Lq,Lk,H,K,D", [
    (1, 70, 2048, 2, 2, 64), (1, 1, 4096, 8, 2, 128), (1, 20, 1024, 160, 160, 64),
    (1, 200, 1500, 4, 2, 128)])
def test_small_probabilities_keep_their_bits(B, Lq, Lk, H, K, D, above, dtype):
    """One key of every 128 lies `above` powers of two over the others and has v = 0. In the
    2-norm the output's own rounding, the probabilities' and that of the f32 sums are each within
    the type's unit."""
    T = R.TYPES[dtype]
    q, k = R.normal(1, (B, Lq, H, D), T), R.normal(2, (B, Lk, K, D), T)
    v = R.normal(3, (B, Lk, K, D), T, 16.0)
    q[..., 0], k[..., 0] = 4.0, 0.0
    k[:, ::128] = 0.0
    k[:, ::128, :, 0] = above * math.log(2.0) * D ** 0.5 / 4.0
    v[:, ::128] = 0.0
    out, lse = fc.attention(q.cuda(), k.cuda(), v.cuda(), return_lse=True)
    want = R.attention(q, k, v)
    ref = want["out"][0]
    off = (out.double().cpu() - ref).norm()
    floor = R.TINY[T] * ref.numel() ** 0.5  # the output's own rounding near zero
    assert off <= 3 * R.U[T] * ref.norm() + floor, float(off / ref.norm() / R.U[T])
    R.check(out, *want["out"], "out")
    R.check(lse, *want["lse"], "lse")
