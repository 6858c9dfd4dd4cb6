"""GPU parity of rotary positions (one to three axes) against the plain 64-bit form, within
bounds derived from the arithmetic (ops_ref)."""
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


def positions(seed, shape, top, dtype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, top, shape, generator=g)
    return p.to(dtype) if dtype != torch.float32 else p.float() + 0.25


CASES = [
    # batch, tokens, heads_q, heads_k, dim, sections
    (1, 1, 1, 1, 2, (1,)), (2, 5, 3, 1, 8, (4,)), (1, 196, 12, 12, 64, (16, 16)),
    (2, 37, 8, 2, 128, (16, 24, 24)), (3, 17, 4, 4, 72, (18, 18)), (1, 9, 2, 2, 80, (10, 15, 15)),
    (2, 11, 5, 5, 33, (7, 9)), (1, 13, 3, 3, 96, (16, 16)), (2, 50, 6, 3, 40, (0, 12, 8)),
    (1, 300, 16, 16, 32, (4, 6, 6)), (1, 7, 40, 8, 256, (64, 64)), (4, 3, 2, 1, 20, (3, 3, 3)),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pairing", ["half", "interleaved", "half_per_axis"])
@pytest.mark.parametrize("B,L,hq,hk,D,sections", CASES)
def test_turns(B, L, hq, hk, D, sections, pairing, dtype):
    T = R.TYPES[dtype]
    q, k = R.normal(1, (B, L, hq, D), T), R.normal(2, (B, L, hk, D), T)
    pos = positions(3, (B, L, len(sections)), 500)
    freq = fc.rope_frequencies(sections, device="cpu")
    for inverse in (False, True):
        a, b = fc.rope(q.cuda(), k.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(),
                       sections=sections, pairing=pairing, inverse=inverse)
        R.check(a, *R.rope(q, pos, freq, sections, pairing, inverse), "q")
        R.check(b, *R.rope(k, pos, freq, sections, pairing, inverse), "k")


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.float32])
def test_position_types_shared_positions_and_long_ones(dtype):
    q = R.normal(4, (2, 40, 3, 64), torch.float32)
    pos = positions(5, (1, 40, 2), 1 << 20, dtype)
    freq = fc.rope_frequencies((16, 16), theta=500000.0, shared=True, device="cpu")
    got = fc.rope(q.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(), sections=(16, 16))
    R.check(got, *R.rope(q, pos, freq, (16, 16), "half"), "q")
    got = fc.rope(q.cuda(), positions=pos[0].cuda(), inv_freq=freq.cuda(), sections=(16, 16))
    R.check(got, *R.rope(q, pos, freq, (16, 16), "half"), "q")
    neg = -pos
    got = fc.rope(q.cuda(), positions=neg.cuda(), inv_freq=freq.cuda(), sections=(16, 16))
    R.check(got, *R.rope(q, neg, freq, (16, 16), "half"), "q")


def test_one_axis_by_default():
    q = R.normal(4, (2, 6, 2, 16), torch.float16)
    pos = positions(5, (6,), 100)
    freq = fc.rope_frequencies((8,), device="cpu")
    got = fc.rope(q.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(), pairing="interleaved")
    R.check(got, *R.rope(q, pos.view(1, 6, 1), freq, (8,), "interleaved"), "q")


@pytest.mark.parametrize("pairing", ["half", "interleaved", "half_per_axis"])
@pytest.mark.parametrize("D,shift", [(64, 0), (64, 1), (72, 0), (30, 3)])
def test_strided_views_in_place_and_guards(pairing, D, shift):
    """q and k inside one wider buffer, head-major or token-major, at aligned and unaligned
    starts; in place nothing else of the buffer changes."""
    B, L, hq, hk = 2, 21, 3, 2
    sections = (D // 8, D // 8, D // 4)
    pos = positions(6, (B, L, 3), 300)
    freq = fc.rope_frequencies(sections, device="cpu")
    for order in ("tokens", "heads"):
        n = B * L * (hq + hk + 1) * D
        buf = R.normal(7, (n + shift + 5,), torch.float16).cuda()
        body = buf[shift:shift + n]
        if order == "tokens":
            whole = body.view(B, L, hq + hk + 1, D)
        else:
            whole = body.view(B, hq + hk + 1, L, D).transpose(1, 2)
        before = buf.clone()
        q, k = whole[:, :, :hq], whole[:, :, hq:hq + hk]
        qc, kc, rest = q.cpu().clone(), k.cpu().clone(), whole[:, :, hq + hk:].clone()
        a, b = fc.rope(q, k, positions=pos.cuda(), inv_freq=freq.cuda(), sections=sections,
                       pairing=pairing)
        assert torch.equal(buf, before)
        R.check(a, *R.rope(qc, pos, freq, sections, pairing), "q")
        R.check(b, *R.rope(kc, pos, freq, sections, pairing), "k")
        fc.rope(q, k, positions=pos.cuda(), inv_freq=freq.cuda(), sections=sections,
                pairing=pairing, out=q, k_out=k)
        assert torch.equal(q, a) and torch.equal(k, b)
        assert torch.equal(whole[:, :, hq + hk:], rest)
        assert torch.equal(buf[:shift], before[:shift]) and torch.equal(buf[-5:], before[-5:])


def test_gradient_is_the_inverse_and_matches_differences():
    """The map is linear: <g, turn(d)> = <turn back(g), d> for every direction d."""
    sections, pairing = (4, 6, 6), "half"
    q, g = R.normal(8, (1, 9, 2, 32), torch.float32), R.normal(9, (1, 9, 2, 32), torch.float32)
    pos = positions(10, (1, 9, 3), 50)
    freq = fc.rope_frequencies(sections, device="cpu")
    got = fc.rope(g.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(), sections=sections,
                  pairing=pairing, inverse=True).double().cpu()
    tol = R.rope(g, pos, freq, sections, pairing, True)[1]
    for seed in range(5):
        d = R.normal(20 + seed, q.shape, torch.float64)
        loss = lambda x: (R_turn(x, pos, freq, sections, pairing) * g.double()).sum()  # noqa
        slope = (loss(q.double() + 1e-3 * d) - loss(q.double() - 1e-3 * d)) / 2e-3
        assert abs((got * d).sum() - slope) <= (tol * d.abs()).sum() + 1e-9 * abs(slope) + 1e-9


def R_turn(x, pos, freq, sections, pairing):
    R.U[torch.float64], R.TINY[torch.float64] = 2.0 ** -53, 0.0
    return R.rope(x, pos, freq, sections, pairing)[0]


def test_empty_stream_and_broadcast_input():
    freq = fc.rope_frequencies((8,), device="cuda")
    q = torch.empty((2, 0, 3, 16), device="cuda")
    pos = torch.empty((2, 0, 1), dtype=torch.int32, device="cuda")
    assert fc.rope(q, positions=pos, inv_freq=freq, sections=(8,)).shape == (2, 0, 3, 16)
    one = R.normal(11, (1, 5, 2, 16), torch.float32)
    pos = positions(12, (3, 5, 1), 90)
    side = torch.cuda.Stream()
    x, p = one.cuda().expand(3, 5, 2, 16), pos.cuda()
    side.wait_stream(torch.cuda.current_stream())
    got = fc.rope(x, positions=p, inv_freq=freq, sections=(8,), stream=side)
    side.synchronize()
    R.check(got, *R.rope(one.expand(3, 5, 2, 16), pos, freq.cpu(), (8,), "half"), "q")


def test_offsets_past_32_bits():
    L, H, D = 300, 2, 16
    far = (1 << 31) + 64
    buf = torch.zeros(far + L * H * D, dtype=torch.float16, device="cuda")
    q = buf.as_strided((2, L, H, D), (far, H * D, D, 1))
    vals = R.normal(13, (2, L, H, D), torch.float16)
    q.copy_(vals.cuda())
    pos = positions(14, (2, L, 1), 1000)
    freq = fc.rope_frequencies((8,), device="cpu")
    fc.rope(q, positions=pos.cuda(), inv_freq=freq.cuda(), sections=(8,), out=q)
    R.check(q, *R.rope(vals, pos, freq, (8,), "half"), "q")
