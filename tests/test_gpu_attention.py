"""GPU parity of attention and its gradient against the plain 64-bit form, within bounds
derived from the arithmetic (ops_ref): types, shared heads, lengths from one token, odd sizes
and head lengths, strides, causal order, ragged and empty sequences, non-finite values in
places that take no part."""
import pytest
import torch

import ops_ref as R
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    yield
    _ops.check_device()


def tensors(B, Lq, Lk, H, K, D, dtype, seed=1):
    T = R.TYPES[dtype]
    return (R.normal(seed, (B, Lq, H, D), T), R.normal(seed + 1, (B, Lk, K, D), T),
            R.normal(seed + 2, (B, Lk, K, D), T), R.normal(seed + 3, (B, Lq, H, D), T))


def lens(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32)


def dev(t):
    return None if t is None else t.cuda()


def run_and_check(q, k, v, g, *, causal=False, scale=None, q_lens=None, kv_lens=None,
                  route="auto", place=None):
    """Forward and backward against the 64-bit form. `place` puts a tensor on the GPU."""
    place = place or dev
    kw = dict(causal=causal, scale=scale, q_lens=dev(q_lens), kv_lens=dev(kv_lens), route=route)
    Q, K, V, Gd = place(q), place(k), place(v), place(g)
    out, lse = fc.attention(Q, K, V, return_lse=True, **kw)
    grads = fc.attention_backward(Gd, Q, K, V, out, lse, **kw)
    want = R.attention(q, k, v, causal=causal, scale=scale, q_lens=q_lens, kv_lens=kv_lens, dout=g)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        R.check(t, *want[name], name)
    return out, lse, grads


SIZES = [
    # B, Lq, Lk, H, K, D
    (1, 1, 1, 1, 1, 64), (2, 1, 300, 4, 4, 64), (1, 1, 1000, 8, 2, 128), (2, 17, 17, 2, 2, 64),
    (1, 196, 196, 3, 3, 64), (2, 64, 128, 2, 1, 32), (1, 129, 257, 2, 2, 128),
    (2, 100, 31, 6, 2, 72), (1, 300, 300, 4, 1, 80), (1, 40, 260, 2, 2, 16), (1, 33, 65, 1, 1, 8),
    (1, 130, 5, 3, 1, 96), (1, 256, 256, 2, 2, 128), (1, 20, 70, 2, 2, 200), (2, 9, 12, 2, 1, 33),
    (1, 5, 9, 1, 1, 1), (1, 50, 90, 10, 2, 120), (1, 385, 513, 1, 1, 64), (1, 3, 129, 12, 4, 64),
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,Lq,Lk,H,K,D", SIZES)
def test_sizes(B, Lq, Lk, H, K, D, dtype, causal):
    run_and_check(*tensors(B, Lq, Lk, H, K, D, dtype), causal=causal)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("B,Lq,Lk,H,K,D", [(2, 70, 70, 2, 1, 64), (1, 33, 140, 4, 2, 128)])
def test_simple_route_in_16_bits(B, Lq, Lk, H, K, D, dtype):
    run_and_check(*tensors(B, Lq, Lk, H, K, D, dtype), causal=True, route="simple")


RAGGED = [
    # causal, q_lens, kv_lens, Lq, Lk
    (False, None, [150, 0, 1, 129], 40, 150), (True, None, [150, 0, 1, 129], 40, 150),
    (True, [150, 0, 1, 129], [150, 0, 1, 129], 150, 150), (False, [0, 7, 40, 13], None, 40, 60),
    (True, [260, 5, 1, 100], [3, 250, 1, 0], 260, 260), (False, [999, -4, 8, 40], [-1, 999, 64, 65], 40, 130),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("causal,ql,kl,Lq,Lk", RAGGED)
@pytest.mark.parametrize("H,K,D", [(4, 2, 64), (3, 3, 128)])
def test_ragged_sequences_with_nan_in_the_padding(causal, ql, kl, Lq, Lk, H, K, D, dtype):
    """Tokens past their lengths hold NaN and infinities and take no part; queries without any
    key give 0, lse -inf and zero gradients."""
    q, k, v, g = tensors(4, Lq, Lk, H, K, D, dtype)
    ql, kl = lens(ql), lens(kl)
    ok = R.allowed(4, Lq, Lk, causal, ql, kl)
    unseen_q, unseen_k = ~ok.any(2), ~ok.any(1)
    q_end = torch.full((4,), Lq) if ql is None else ql.clamp(0, Lq)
    k_end = torch.full((4,), Lk) if kl is None else kl.clamp(0, Lk)
    for b in range(4):
        for t in (q, g):
            t[b, int(q_end[b]):] = NAN
            t[b, int(q_end[b]):][::2] = float("inf")
        for t in (k, v):
            t[b, int(k_end[b]):] = NAN
            t[b, int(k_end[b]):][::2] = float("-inf")
    out, lse, (dq, dk, dv) = run_and_check(q, k, v, g, causal=causal, q_lens=ql, kv_lens=kl)
    out, lse, dq, dk, dv = (t.cpu() for t in (out, lse, dq, dk, dv))
    assert torch.count_nonzero(out[unseen_q]) == 0 and torch.count_nonzero(dq[unseen_q]) == 0
    assert (lse.transpose(1, 2)[unseen_q] == -float("inf")).all()
    assert torch.count_nonzero(dk[unseen_k]) == 0 and torch.count_nonzero(dv[unseen_k]) == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_nan_in_queries_that_see_no_key(dtype):
    """Causal order with more queries than keys: the first queries see nothing; NaN there does
    not reach the keys' gradients."""
    q, k, v, g = tensors(1, 200, 60, 2, 2, 64, dtype)
    q[:, :140], g[:, :140] = NAN, NAN
    run_and_check(q, k, v, g, causal=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "heads_first", "odd", "broadcast"])
@pytest.mark.parametrize("D", [64, 72, 128])
def test_strides(layout, D, dtype):
    """Views of a fused projection, head-major tensors, rows of an odd length at an odd start,
    and keys broadcast over the batch; outputs given as strided views with guards."""
    T = R.TYPES[dtype]
    B, L, H, K = 2, 150, 4, 2
    q, k, v, g = tensors(B, L, L, H, K, D, dtype)
    if layout == "broadcast":
        k, v = k[:1].expand(B, L, K, D), v[:1].expand(B, L, K, D)

    def place(t):
        if layout == "heads_first":
            return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        if layout == "odd":
            b = torch.full((t.shape[0], t.shape[1], t.shape[2], D + 3), NAN, dtype=T, device="cuda")
            b[..., 1:D + 1] = t.cuda()
            return b[..., 1:D + 1]
        if layout == "broadcast" and t.shape[2] == K:
            return t[:1].contiguous().cuda().expand(t.shape)
        wide = torch.full((t.shape[0], t.shape[1], t.shape[2] + 3, D), NAN, dtype=T, device="cuda")
        wide[:, :, 1:-2] = t.cuda()
        return wide[:, :, 1:-2]

    Q, Kd, V, G = place(q), place(k), place(v), place(g)
    wide = torch.full((B, L, H + 2 * K + 2, D), 7.0, dtype=T, device="cuda")
    dq, dk, dv = wide[:, :, 1:H + 1], wide[:, :, H + 1:H + K + 1], wide[:, :, H + K + 1:-1]
    obuf = torch.full((B, H, L, D + 8), 7.0, dtype=T, device="cuda")
    o = obuf[..., :D].transpose(1, 2)
    out, lse = fc.attention(Q, Kd, V, causal=True, return_lse=True, out=o)
    fc.attention_backward(G, Q, Kd, V, out, lse, causal=True, dq=dq, dk=dk, dv=dv)
    want = R.attention(q, k, v, causal=True, dout=g)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (o, lse, dq, dk, dv)):
        R.check(t, *want[name], name)
    assert (obuf[..., D:] == 7).all() and (wide[:, :, 0] == 7).all() and (wide[:, :, -1] == 7).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,Lq,Lk,H,K,D,causal", [
    (1, 1, 5000, 8, 1, 128, False), (3, 1, 2500, 4, 4, 64, False), (1, 2, 4096, 16, 2, 128, True),
    (1, 7, 3001, 4, 4, 72, True), (2, 130, 1900, 2, 2, 64, False), (1, 1, 8000, 1, 1, 64, False)])
def test_few_queries_over_long_sequences(B, Lq, Lk, H, K, D, causal, dtype):
    """One to a few query tokens: the keys are split over many blocks and joined."""
    q, k, v, g = tensors(B, Lq, Lk, H, K, D, dtype)
    kl = lens([max(0, Lk - 777 * b) for b in range(B)])
    run_and_check(q, k, v, g, causal=causal, kv_lens=kl)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_scores_of_every_size(dtype):
    """A scale that makes the softmax nearly one-hot, rows whose maximum grows along the keys
    (every tile rescales) and a scale near zero."""
    q, k, v, g = tensors(1, 70, 600, 2, 2, 64, dtype)
    run_and_check(q, k, v, g, scale=2.0)
    ramp = (torch.arange(600) / 600.0 * 4.0).to(k.dtype)
    k2 = k * ramp[None, :, None, None]
    run_and_check(q, k2, v, g, scale=1.0)
    run_and_check(q, k2.flip(1).contiguous(), v, g, scale=1.0)
    run_and_check(q, k, v, g, scale=1e-6)


def test_infinite_scores():
    """Keys of the type's lowest value give scores that round to -inf: probability zero."""
    q, k, v, g = tensors(1, 20, 150, 2, 2, 64, "f32")
    q = q.abs() + 0.5
    k[:, 10:90] = -3.0e38
    out, lse = fc.attention(q.cuda(), k.cuda(), v.cuda(), return_lse=True)
    keep = [i for i in range(150) if not 10 <= i < 90]
    want = R.attention(q, k[:, keep], v[:, keep])
    R.check(out, *want["out"], "out")
    R.check(lse, *want["lse"], "lse")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_empty_extents(dtype):
    T = R.TYPES[dtype]
    e = lambda *s: torch.ones(s, dtype=T, device="cuda")  # noqa: E731
    out, lse = fc.attention(e(2, 5, 4, 64), e(2, 0, 2, 64), e(2, 0, 2, 64), return_lse=True)
    assert torch.count_nonzero(out) == 0 and (lse == -float("inf")).all()
    dq, dk, dv = fc.attention_backward(e(2, 5, 4, 64), e(2, 5, 4, 64), e(2, 0, 2, 64),
                                       e(2, 0, 2, 64), out, lse)
    assert torch.count_nonzero(dq) == 0 and dk.numel() == 0
    out, lse = fc.attention(e(2, 0, 4, 64), e(2, 7, 2, 64), e(2, 7, 2, 64), return_lse=True)
    assert out.shape == (2, 0, 4, 64)
    dq, dk, dv = fc.attention_backward(out, out, e(2, 7, 2, 64), e(2, 7, 2, 64), out, lse)
    assert torch.count_nonzero(dk) == 0 and torch.count_nonzero(dv) == 0
    assert fc.attention(e(0, 3, 4, 64), e(0, 7, 2, 64), e(0, 7, 2, 64)).shape == (0, 3, 4, 64)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_repeats_streams_and_alone_forward(dtype):
    """The same call gives the same bits, on another stream too, with and without lse."""
    q, k, v, g = (t.cuda() for t in tensors(2, 200, 333, 8, 2, 64, dtype))
    out, lse = fc.attention(q, k, v, return_lse=True)
    grads = fc.attention_backward(g, q, k, v, out, lse)
    assert torch.equal(out, fc.attention(q, k, v))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = fc.attention(q, k, v, return_lse=True, stream=side)
    g2 = fc.attention_backward(g, q, k, v, o2, l2, stream=side)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    for a, b in zip(grads, g2):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """Directional differences of the 64-bit loss, within the gradient's own bounds."""
    q, k, v, g = tensors(1, 12, 19, 4, 2, 16, "f32")
    kw = dict(causal=True, kv_lens=lens([17]))
    out, lse = fc.attention(q.cuda(), k.cuda(), v.cuda(), return_lse=True, causal=True,
                            kv_lens=kw["kv_lens"].cuda())
    got = fc.attention_backward(g.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, causal=True,
                                kv_lens=kw["kv_lens"].cuda())
    want = R.attention(q, k, v, dout=g, **kw)
    R.U[torch.float64], R.TINY[torch.float64] = 2.0 ** -53, 0.0
    loss = lambda *a: (R.attention(*a, **kw)["out"][0] * g.double()).sum()  # noqa: E731
    args = [q.double(), k.double(), v.double()]
    for i, name in enumerate(("dq", "dk", "dv")):
        for seed in range(3):
            d = R.normal(50 + seed, args[i].shape, torch.float64)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + 1e-4 * d, args[i] - 1e-4 * d
            slope = (loss(*up) - loss(*down)) / 2e-4
            dot = (got[i].double().cpu() * d).sum()
            assert abs(dot - slope) <= (want[name][1] * d.abs()).sum() + 1e-6 * abs(slope) + 1e-7


@pytest.mark.parametrize("dtype", ["f16"])
def test_offsets_past_32_bits(dtype):
    """Sequences more than 2^31 elements apart."""
    B, L, H, D = 2, 140, 2, 64
    q, k, v, g = tensors(B, L, L, H, H, D, dtype)
    far = (1 << 31) + 256

    def place(t):
        buf = torch.zeros(far + L * H * D, dtype=t.dtype, device="cuda")
        x = buf.as_strided((B, L, H, D), (far, H * D, D, 1))
        x.copy_(t.cuda())
        return x

    run_and_check(q, k, v, g, causal=True, place=place)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -13, 1.0, 256.0])
def test_gradients_of_every_size(dtype, size):
    """Small output gradients over long sequences (score gradients far below f16's smallest
    normal value) and large ones (score gradients past f16's largest value times the keys)
    keep the relative accuracy of the type."""
    q, k, v, g = tensors(1, 260, 1300, 2, 1, 64, dtype)
    T = R.TYPES[dtype]
    g, v = (g.float() * size).to(T), (v.float() * 8).to(T)
    out, lse = fc.attention(q.cuda(), k.cuda(), v.cuda(), return_lse=True)
    got = fc.attention_backward(g.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse)
    want = R.attention(q, k, v, dout=g)
    for name, t in zip(("dq", "dk", "dv"), got):
        ref = want[name][0]
        floor = R.TINY[T] * ref.numel() ** 0.5  # the output's own rounding near zero
        off = (t.double().cpu() - ref).norm()
        assert off <= 3 * R.U[T] * ref.norm() + floor, (name, float(off / ref.norm()))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_many_tiles_and_items_a_block(D, causal):
    """More work items than SMs, each of many tiles, so that every block's rings, phases and
    accumulators go round many times: two heads of one head's data give the same bits, and a
    head computed alone agrees with it."""
    B, L, H = 2, 1700, 48
    q, k, v, g = tensors(B, L, L, 1, 1, D, "bf16")
    rep = lambda t: t.cuda().expand(B, L, H, D).contiguous()  # noqa: E731
    kl = lens([1700, 901]).cuda()
    out, lse = fc.attention(rep(q), rep(k), rep(v), causal=causal, kv_lens=kl, return_lse=True)
    grads = fc.attention_backward(rep(g), rep(q), rep(k), rep(v), out, lse, causal=causal,
                                  kv_lens=kl)
    one, l1 = fc.attention(q.cuda(), k.cuda(), v.cuda(), causal=causal, kv_lens=kl,
                           return_lse=True, route="simple")
    g1 = fc.attention_backward(g.cuda(), q.cuda(), k.cuda(), v.cuda(), one, l1, causal=causal,
                               kv_lens=kl, route="simple")
    for name, many, single in zip(("out", "dq", "dk", "dv"), (out, *grads), (one, *g1)):
        assert torch.equal(many, many[:, :, :1].expand_as(many)), name
        a, b = many[:, :, :1].double(), single.double()
        assert (a - b).norm() <= 4 * R.U[torch.bfloat16] * b.norm(), name
    assert torch.equal(lse, lse[:, :1].expand_as(lse))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,Lq,Lk,H,K,D,causal,kl", [
    (2, 70, 200, 4, 2, 256, True, [200, 65]), (1, 129, 129, 2, 2, 136, False, None),
    (3, 33, 97, 3, 1, 192, False, [97, 0, 31]), (1, 1, 300, 8, 2, 256, True, None),
    (2, 100, 40, 2, 1, 129, True, [40, 7]), (1, 65, 65, 1, 1, 251, True, None),
])
def test_head_lengths_over_128(B, Lq, Lk, H, K, D, causal, kl, dtype):
    """Odd lengths, rows that are whole 16-byte units and ones that are not, several tiles of
    queries and keys, keys cut short, queries without a key."""
    run_and_check(*tensors(B, Lq, Lk, H, K, D, dtype), causal=causal, kv_lens=lens(kl))
