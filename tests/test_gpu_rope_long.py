"""Rotary positions past what an f32 holds exactly, against the plain 64-bit form. The
frequencies are such that the form's own products are exact (53 bits)."""
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


def odd(seed, low, high, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(low, high, shape, generator=g) | 1).to(dtype)


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("sign", [1, -1])
def test_integers_up_to_2_29(pairing, dtype, sign):
    q = R.normal(1, (2, 50, 3, 64), torch.float32)
    pos = sign * odd(2, 1 << 24, 1 << 29, (2, 50, 2), dtype)
    freq = fc.rope_frequencies((16, 16), theta=500000.0, device="cpu")
    got = fc.rope(q.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(), sections=(16, 16),
                  pairing=pairing)
    R.check(got, *R.rope(q, pos, freq, (16, 16), pairing), "q")


@pytest.mark.parametrize("dtype,low,high", [
    (torch.int32, (1 << 31) - 5000, (1 << 31) - 1), (torch.int64, 1 << 40, 1 << 41),
    (torch.int64, 1 << 52, 1 << 53), (torch.float32, 1 << 24, 1 << 40)])
def test_longest_positions(dtype, low, high):
    """Frequencies that are powers of two."""
    q = R.normal(3, (1, 80, 2, 32), torch.float32)
    pos = odd(4, low, high, (1, 80, 1), torch.int64).to(dtype)
    freq = 2.0 ** -torch.arange(16, dtype=torch.float32)
    got = fc.rope(q.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(), sections=(16,))
    R.check(got, *R.rope(q, pos, freq, (16,), "half"), "q")


def test_short_and_long_positions_mixed():
    """Around the size where the products change their form, neighbours agree with 64 bits."""
    pos = torch.cat([torch.arange((1 << s) - 20, (1 << s) + 20) for s in (10, 22, 23, 24, 25)])
    q = R.normal(5, (1, len(pos), 2, 32), torch.float32)
    freq = fc.rope_frequencies((16,), device="cpu")
    for p in (pos.int(), pos):
        got = fc.rope(q.cuda(), positions=p.cuda(), inv_freq=freq.cuda(), sections=(16,))
        R.check(got, *R.rope(q, p.view(1, -1, 1), freq, (16,), "half"), "q")
