"""Sums of the gated block over more products than one accumulator of the tensor cores should take:
they cut off what passes f32, always towards zero. All values are positive here, so that nothing of
that cancels: without passes whose sums are added in plain f32 the weights' gradients of 2^18 tokens
came out 1.7e-3 too small, 3.5 times f16's rounding."""
import math

import pytest
import torch

from ops_ref import E32, U
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dw_gate", "dw_up", "dw_down")


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    yield
    _ops.check_device()


def cut(K):
    """What a sum of K positive products loses on tensor cores: an instruction of 16 cuts its products
    and the sum at the sum's last place, 4 units of the sum so far at the most (1.7 on average,
    measured), and that is half of the whole sum on average; passes are of 16384 at the most."""
    return 2 * E32 * min(K, 16384) / 16 + (K / 16384 + 8) * E32


def carried(e, K, u):
    """What operands that are too small by e of themselves before they are rounded do to a sum of K
    of them: e on average, by roundings that fall to the other side. Those come with probability
    e / (2 u) at the most, independently, and move a term by one step, 2 u of it at the most: six
    times the standard deviation of their mean, a quarter more for terms of unequal size."""
    return e + 6 * 1.25 * 2 * u * math.sqrt(min(1.0, e / (2 * u)) / K)


def check(got, ref, rel, what):
    far = ((got.double() - ref).abs() / ref).max().item()
    assert far <= rel, f"{what}: {far:.2e} of the value, bound {rel:.2e}"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,c,f,o", [
    (1 << 18, 64, 64, 64),      # long weight gradients of one tile each
    (40000, 1541, 1536, 1544),  # of many tiles, some by rows
    (2600, 40000, 1544, 64),    # a long gated product
    (300, 40000, 264, 24),
    (2600, 64, 40000, 1544),    # long down projection and dx
    (300, 24, 40000, 264),
    (2600, 64, 1544, 40000),    # a long gradient of the hidden values
    (40, 17000, 17000, 40),     # blocks that share a tile
])
def test_long_sums_of_positive_values(n, c, f, o, dtype):
    g = torch.Generator(device="cuda").manual_seed(n + c)

    def positive(*shape, scale=1.0):
        return (torch.rand(shape, generator=g, device="cuda") + 0.25).mul_(scale).to(dtype)

    # powers of two that keep the results of f16, too, within its normal range
    bits = c.bit_length() - 1
    x, wg, wu = (positive(*shape, scale=2.0 ** -k) for shape, k in
                 (((n, c), bits // 2), ((f, c), bits - bits // 2), ((f, c), bits - bits // 2)))
    wd, dy = positive(o, f, scale=2.0 ** -9), positive(n, o, scale=2.0 ** round(math.log2(5 / o)))
    y, saved = fc.gated_mlp(x, wg, wu, wd, activation=None, return_saved=True)
    grads = dict(zip(NAMES, fc.gated_mlp_backward(dy, x, wg, wu, wd, saved, activation=None)))

    X, G, UP, D, DY = (t.double() for t in (x, wg, wu, wd, dy))
    gate, up, dh = X @ G.t(), X @ UP.t(), DY @ D
    h, dg, du = ((a * b).to(dtype).double() for a, b in ((gate, up), (dh, up), (dh, gate)))
    # operands: what the sums they come from lose
    eh, ed = 2 * cut(c) + 8 * E32, cut(c) + cut(o) + 8 * E32
    u = U[dtype]
    check(y, h @ D.t(), 1.05 * u + carried(eh, f, u) + cut(f), "y")
    check(grads["dx"], dg @ G + du @ UP, 1.05 * u + carried(ed, 2 * f, u) + cut(2 * f), "dx")
    check(grads["dw_gate"], dg.t() @ X, 1.05 * u + carried(ed, n, u) + cut(n), "dw_gate")
    check(grads["dw_up"], du.t() @ X, 1.05 * u + carried(ed, n, u) + cut(n), "dw_up")
    check(grads["dw_down"], DY.t() @ h, 1.05 * u + carried(eh, n, u) + cut(n), "dw_down")
    for t in (y, *grads.values()):
        assert torch.isfinite(t).all()
