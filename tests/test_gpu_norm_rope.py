"""GPU parity of the head norms with rotation, forward and backward, against the plain 64-bit
forms, within bounds derived from the arithmetic (block_ref)."""
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


def positions(seed, shape, top, dtype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, top, shape, generator=g).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


def case(seed, b, n, hq, hk, d, sections, T, P):
    q, dq = R.normal(seed, (b, n, hq, d), T, 1.7), R.normal(seed + 1, (b, n, hq, d), T)
    k = dk = kw = None
    if hk:
        k, dk = R.normal(seed + 2, (b, n, hk, d), T, 0.6), R.normal(seed + 3, (b, n, hk, d), T)
        kw = R.normal(seed + 5, (d,), P, 0.2, 1.0)
    w = R.normal(seed + 4, (d,), P, 0.2, 1.0)
    pos = freq = None
    if sections:
        pos = positions(seed + 6, (b, n, len(sections)), 700)
        freq = fc.rope_frequencies(sections, device="cpu")
    return q, k, w, kw, pos, freq, dq, dk


def check_both(q, k, w, kw, pos, freq, dq, dk, sections, pairing, eps=1e-6):
    how = dict(weight=cuda(w), k_weight=cuda(kw), positions=cuda(pos), inv_freq=cuda(freq),
               sections=sections, pairing=pairing, eps=eps)
    got = fc.norm_rope(cuda(q), cuda(k), **how)
    got = (got, None) if k is None else got
    grads = fc.norm_rope_backward(cuda(dq), cuda(q), cuda(dk), cuda(k), **how)
    for x, wt, dy, y, dx, dw in ((q, w, dq, got[0], grads[0], grads[2]),
                                 (k, kw, dk, got[1], grads[1], grads[3])):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        R.check(y, *B.norm_rope(x, wt, pos, freq, sections, pairing, eps), "y")
        ref = B.norm_rope_backward(dy, x, wt, pos, freq, sections, pairing, eps)
        R.check(dx, *ref["dx"], "dx")
        if wt is not None:
            R.check(dw, *ref["dw"], "dw")


CASES = [
    # batch, tokens, heads_q, heads_k, dim, sections
    (1, 1, 1, 1, 2, (1,)), (2, 5, 3, 1, 8, (4,)), (1, 196, 12, 12, 64, (16, 16)),
    (2, 37, 8, 2, 128, (16, 24, 24)), (3, 17, 4, 4, 72, (18, 18)), (1, 9, 2, 2, 80, (10, 15, 15)),
    (2, 11, 5, 5, 33, (7, 9)), (1, 13, 3, 0, 96, (16, 16)), (2, 50, 6, 3, 40, (0, 12, 8)),
    (1, 70, 16, 16, 32, (4, 6, 6)), (1, 7, 40, 8, 256, (64, 64)), (4, 3, 2, 1, 20, (3, 3, 3)),
    (1, 6, 3, 2, 512, (128, 128)), (2, 5, 2, 1, 511, (200,)), (1, 9, 2, 2, 300, (75, 75)),
    (2, 8, 4, 2, 128, (32,)), (1, 12, 3, 3, 64, None), (1, 3, 2, 1, 1, None),
    (1, 40, 2, 2, 48, (8, 8)),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pairing", ["half", "interleaved", "half_per_axis"])
@pytest.mark.parametrize("b,n,hq,hk,d,sections", CASES)
def test_forward_and_backward(b, n, hq, hk, d, sections, pairing, dtype):
    T = R.TYPES[dtype]
    P = torch.float32 if (hq + n) % 2 else T  # both types of weights over the cases
    check_both(*case(100, b, n, hq, hk, d, sections, T, P), sections, pairing)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_weights_and_with_one(dtype):
    q, k, w, kw, pos, freq, dq, dk = case(200, 2, 19, 4, 2, 64, (16, 16), R.TYPES[dtype],
                                          R.TYPES[dtype])
    for a, b in ((None, None), (w, None), (None, kw)):
        check_both(q, k, a, b, pos, freq, dq, dk, (16, 16), "half")


@pytest.mark.parametrize("n", [1500, 9000])
def test_blocks_that_take_many_tokens(n):
    """More tokens than the backward pass has lanes, so that its blocks go round."""
    check_both(*case(300, 2, n, 3, 1, 64, (32,), torch.float16, torch.float32), (32,), "half")


def test_zero_rows_and_eps():
    """A head of zeros stays zero, and its gradient is finite: dy w / sqrt(eps)."""
    q, k, w, kw, pos, freq, dq, dk = case(400, 1, 7, 2, 1, 64, (32,), torch.float32, torch.float32)
    q[0, 3, 1] = 0.0
    k[0, :, 0] *= 1e-4
    check_both(q, k, w, kw, pos, freq, dq, dk, (32,), "half", eps=1e-5)


def test_non_finite_heads_stay_by_themselves():
    q, k, w, kw, pos, freq, dq, dk = case(500, 1, 20, 4, 2, 128, (64,), torch.bfloat16,
                                          torch.bfloat16)
    how = dict(weight=w.cuda(), k_weight=kw.cuda(), positions=pos.cuda(), inv_freq=freq.cuda())
    clean = fc.norm_rope(q.cuda(), k.cuda(), **how)
    q[0, 5, 2, 7], k[0, 9, 1, 100] = float("nan"), float("inf")
    got = fc.norm_rope(q.cuda(), k.cuda(), **how)
    for a, b, at in ((clean[0], got[0], (0, 5, 2)), (clean[1], got[1], (0, 9, 1))):
        same = (a == b).all(-1)
        assert not same[at] and int((~same).sum()) == 1
    # elements without a pair are not mixed with each other
    x = R.normal(7, (1, 2, 1, 16), torch.float32)
    x[0, 1, 0, 15] = float("inf")
    y = fc.norm_rope(x.cuda(), positions=torch.zeros(2, 1, dtype=torch.int32).cuda(),
                     inv_freq=torch.ones(4).cuda(), sections=(4,)).cpu()
    assert torch.isnan(y[0, 1, 0, 15]) and (y[0, 1, 0, :15] == 0).all()


@pytest.mark.parametrize("pairing", ["half", "interleaved", "half_per_axis"])
@pytest.mark.parametrize("d,shift", [(64, 0), (64, 1), (72, 4), (30, 3)])
def test_strided_views_in_place_and_guards(pairing, d, shift):
    b, n, hq, hk = 2, 21, 3, 2
    sections = (d // 8, d // 8, d // 4)
    q, k, w, kw, pos, freq, dq, dk = case(600, b, n, hq, hk, d, sections, torch.float16,
                                          torch.float16)
    how = dict(weight=w.cuda(), k_weight=kw.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(),
               sections=sections, pairing=pairing)
    for order in ("tokens", "heads"):
        size = b * n * (hq + hk + 1) * d

        def fill(a, c):
            buf = R.normal(7, (size + shift + 5,), torch.float16).cuda()
            body = buf[shift:shift + size]
            whole = body.view(b, n, hq + hk + 1, d) if order == "tokens" else \
                body.view(b, hq + hk + 1, n, d).transpose(1, 2)
            whole[:, :, :hq], whole[:, :, hq:hq + hk] = a.cuda(), c.cuda()
            return buf, whole, whole[:, :, :hq], whole[:, :, hq:hq + hk]

        buf, whole, qs, ks = fill(q, k)
        gbuf, gwhole, dqs, dks = fill(dq, dk)
        before, gbefore = buf.clone(), gbuf.clone()
        y = fc.norm_rope(qs, ks, **how)
        grads = fc.norm_rope_backward(dqs, qs, dks, ks, **how)
        assert torch.equal(buf, before) and torch.equal(gbuf, gbefore)
        for x, wt, dy, out, dx, dw in ((q, w, dq, y[0], grads[0], grads[2]),
                                       (k, kw, dk, y[1], grads[1], grads[3])):
            R.check(out, *B.norm_rope(x, wt, pos, freq, sections, pairing, 1e-6), "y")
            ref = B.norm_rope_backward(dy, x, wt, pos, freq, sections, pairing, 1e-6)
            R.check(dx, *ref["dx"], "dx")
            R.check(dw, *ref["dw"], "dw")
        # in place: nothing else of the buffers changes
        again = fc.norm_rope_backward(dqs, qs, dks, ks, **how, dq=dqs, dk=dks)
        fc.norm_rope(qs, ks, **how, out=qs, k_out=ks)
        for a, c in ((qs, y[0]), (ks, y[1]), (dqs, grads[0]), (dks, grads[1]),
                     (again[2], grads[2]), (again[3], grads[3])):
            assert torch.equal(a, c)
        for now, was, tail, old in ((buf, before, whole, None), (gbuf, gbefore, gwhole, None)):
            assert torch.equal(now[:shift], was[:shift]) and torch.equal(now[-5:], was[-5:])
            rest = was[shift:shift + size]
            rest = rest.view(b, n, hq + hk + 1, d) if order == "tokens" else \
                rest.view(b, hq + hk + 1, n, d).transpose(1, 2)
            assert torch.equal(tail[:, :, hq + hk:], rest[:, :, hq + hk:])


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.float32])
def test_position_types_long_positions_and_broadcast_rows(dtype):
    x = R.normal(4, (1, 40, 3, 64), torch.float32)
    pos = positions(5, (40, 2), 1 << 20, dtype)
    freq = fc.rope_frequencies((16, 16), theta=500000.0, shared=True, device="cpu")
    got = fc.norm_rope(x.cuda().expand(2, 40, 3, 64), positions=pos.cuda(), inv_freq=freq.cuda(),
                       sections=(16, 16))
    R.check(got, *B.norm_rope(x.expand(2, 40, 3, 64), None, pos, freq, (16, 16), "half", 1e-6), "y")
    if dtype == torch.int64:
        # 41 bits times the 24 of a frequency would round in 64 bits, by up to 2^-13: powers of two
        far, freq = pos + (1 << 40), 2.0 ** -torch.arange(32, dtype=torch.float32)
        got = fc.norm_rope(x.cuda(), positions=far.cuda(), inv_freq=freq.cuda(), sections=(16, 16))
        R.check(got, *B.norm_rope(x, None, far, freq, (16, 16), "half", 1e-6), "y")


def test_no_tokens():
    w = torch.ones(16, device="cuda")
    q = torch.empty((2, 0, 3, 16), device="cuda")
    assert fc.norm_rope(q, weight=w).shape == q.shape
    dq, dk, dw, dkw = fc.norm_rope_backward(q, q, weight=w)
    assert dq.shape == q.shape and dk is None and dkw is None and (dw == 0).all()


def test_gradient_matches_differences():
    """Central differences of a 64-bit loss along random directions."""
    q, _, w, _, pos, freq, dq, _ = case(700, 1, 9, 2, 0, 32, (4, 6, 6), torch.float32,
                                        torch.float32)
    dx, _, dw, _ = (cuda(t) for t in fc.norm_rope_backward(
        dq.cuda(), q.cuda(), weight=w.cuda(), positions=pos.cuda(), inv_freq=freq.cuda(),
        sections=(4, 6, 6)))

    def loss(x, wt):
        r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        return (B._turn(x * r * wt, pos, freq, (4, 6, 6), "half")[0] * dq.double()).sum()

    ref = B.norm_rope_backward(dq, q, w, pos, freq, (4, 6, 6), "half", 1e-6)
    for seed in range(4):
        d, e = R.normal(20 + seed, q.shape, torch.float64), R.normal(30 + seed, w.shape, torch.float64)
        t = 1e-4
        slope = (loss(q.double() + t * d, w.double() + t * e)
                 - loss(q.double() - t * d, w.double() - t * e)) / (2 * t)
        got = (dx.double().cpu() * d).sum() + (dw.double().cpu() * e).sum()
        tol = (ref["dx"][1] * d.abs()).sum() + (ref["dw"][1] * e.abs()).sum()
        assert abs(got - slope) <= tol + 1e-5 * abs(slope) + 1e-5


def test_streams_and_a_captured_graph():
    """On another stream, and captured twice into one graph with results that repeat bit by bit."""
    q, k, w, kw, pos, freq, dq, dk = (cuda(t) for t in case(800, 2, 333, 8, 2, 128, (64,),
                                                            torch.bfloat16, torch.bfloat16))
    how = dict(weight=w, k_weight=kw, positions=pos, inv_freq=freq)

    def both(stream=None):
        return (*fc.norm_rope(q, k, **how, stream=stream),
                *fc.norm_rope_backward(dq, q, dk, k, **how, stream=stream))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one, two = both(), both()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got in (other, one, two):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    n, h, d = 300, 2, 16
    far = (1 << 31) + 64
    buf = torch.zeros(far + n * h * d, dtype=torch.float16, device="cuda")
    q = buf.as_strided((2, n, h, d), (far, h * d, d, 1))
    vals = R.normal(13, (2, n, h, d), torch.float16)
    q.copy_(vals.cuda())
    fc.norm_rope(q, out=q)
    R.check(q, *B.norm_rope(vals, None, None, None, None, "half", 1e-6), "y")
