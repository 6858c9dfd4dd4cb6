"""Attention in f32 at the ends of the type: its lowest and largest values and infinities in
queries, keys, values and output gradients."""
import pytest
import torch

import ops_ref as R
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu
LOWEST, LARGEST = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
INF = float("inf")
SIZES = [(1, 20, 150, 2, 2, 64), (2, 70, 90, 4, 2, 72), (1, 33, 140, 2, 1, 33),
         (1, 40, 100, 2, 2, 200)]


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    yield
    _ops.check_device()


def tensors(B, Lq, Lk, H, K, D):
    q, g = (R.normal(s, (B, Lq, H, D), torch.float32) for s in (1, 4))
    k, v = (R.normal(s, (B, Lk, K, D), torch.float32) for s in (2, 3))
    return q, k, v, g


def run(q, k, v, g, **kw):
    Q, K, V, G = (t.cuda() for t in (q, k, v, g))
    out, lse = fc.attention(Q, K, V, return_lse=True, **kw)
    return (out, lse, *fc.attention_backward(G, Q, K, V, out, lse, **kw))


@pytest.mark.parametrize("value", [LOWEST, -3.0e38, -INF])
@pytest.mark.parametrize("B,Lq,Lk,H,K,D", SIZES)
def test_keys_of_the_lowest_value(B, Lq, Lk, H, K, D, value):
    """Queries of one sign meet keys of the type's lowest value (or minus infinity): their scores
    are -inf, their probabilities 0, and all else is as if they were not there."""
    q, k, v, g = tensors(B, Lq, Lk, H, K, D)
    q = q.abs() + 0.5
    hidden = torch.zeros(Lk, dtype=torch.bool)
    hidden[3:40] = hidden[Lk - 5] = True
    k[:, hidden] = value
    out, lse, dq, dk, dv = run(q, k, v, g)
    want = R.attention(q, k[:, ~hidden], v[:, ~hidden], dout=g)
    R.check(out, *want["out"], "out")
    R.check(lse, *want["lse"], "lse")
    R.check(dk[:, ~hidden], *want["dk"], "dk")
    R.check(dv[:, ~hidden], *want["dv"], "dv")
    assert torch.count_nonzero(dk[:, hidden]) == 0 and torch.count_nonzero(dv[:, hidden]) == 0
    if value != -INF:  # the sum over the keys has 0 * inf in it otherwise
        R.check(dq, *want["dq"], "dq")


@pytest.mark.parametrize("B,Lq,Lk,H,K,D", SIZES)
def test_values_of_the_largest_size_and_infinite(B, Lq, Lk, H, K, D):
    q, k, v, g = tensors(B, Lq, Lk, H, K, D)
    v[:, 7, :, 3], v[:, 9, :, 5], v[:, 11, :, 6] = LARGEST, LOWEST, 3.403e38 * 0.9999
    Q, Kd, V = q.cuda(), k.cuda(), v.cuda()
    out = fc.attention(Q, Kd, V)
    R.check(out, *R.attention(q, k, v)["out"], "out")
    v[:, 7, :, 3], v[:, 9, :, 5] = INF, -INF
    got = fc.attention(Q, Kd, v.cuda()).cpu()
    want = R.attention(q, k, v)["out"][0]
    assert (got[..., 3] == INF).all() and (got[..., 5] == -INF).all()
    assert (want[..., 3] == INF).all() and (want[..., 5] == -INF).all()
    rest = [d for d in range(D) if d not in (3, 5)]
    assert torch.equal(got[..., rest], out.cpu()[..., rest])


@pytest.mark.parametrize("B,Lq,Lk,H,K,D", SIZES)
def test_output_gradients_of_the_largest_size(B, Lq, Lk, H, K, D):
    q, k, v, g = tensors(B, Lq, Lk, H, K, D)
    v = v * 2.0 ** -10
    g[:, 3, :, 5], g[:, 5, :, 1] = LARGEST, LOWEST
    out, lse, dq, dk, dv = run(q, k, v, g)
    want = R.attention(q, k, v, dout=g)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        R.check(t, *want[name], name)


@pytest.mark.parametrize("B,Lq,Lk,H,K,D", SIZES)
def test_queries_of_the_largest_size(B, Lq, Lk, H, K, D):
    """A query of the largest value against keys of 2^-100, whose remainders past TF32 are still
    normal numbers; the scale brings the scores to ordinary sizes."""
    q, k, v, g = tensors(B, Lq, Lk, H, K, D)
    q[:, 2] = 0.0
    q[:, 2, :, 1], q[:, 4] = LARGEST, q[:, 4] * 2.0 ** 126
    k = k * 2.0 ** -100
    out, lse = fc.attention(q.cuda(), k.cuda(), v.cuda(), scale=2.0 ** -28, return_lse=True)
    want = R.attention(q, k, v, scale=2.0 ** -28)
    R.check(out, *want["out"], "out")
    R.check(lse, *want["lse"], "lse")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("route", ["auto", "simple"])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_only_scores_of_minus_infinity(D, route, dtype):
    """Every score of a sequence is -inf: its rows have out 0, lse -inf and no gradient, and the
    other sequence is not touched."""
    T = R.TYPES[dtype]
    q, k, v, g = (t.to(T) for t in tensors(2, 70, 150, 4, 2, D))
    q = q.abs() + 0.5
    k[1] = -3.0e38
    out, lse, dq, dk, dv = run(q, k, v, g, route=route)
    want = R.attention(q[:1], k[:1], v[:1], dout=g[:1])
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, dq, dk, dv)):
        R.check(t[:1], *want[name], name)
    assert (lse[1] == -INF).all()
    for t in (out, dq, dk, dv):
        assert torch.count_nonzero(t[1]) == 0


@pytest.mark.parametrize("B,Lq,Lk,H,K,D", SIZES)
def test_keys_and_values_of_the_lowest_value(B, Lq, Lk, H, K, D):
    """Slots filled with the lowest value in keys and values alike: probability 0, although the
    product of the output gradient with such a value is not finite."""
    q, k, v, g = tensors(B, Lq, Lk, H, K, D)
    q = q.abs() + 0.5
    hidden = torch.zeros(Lk, dtype=torch.bool)
    hidden[10:30] = True
    k[:, hidden], v[:, hidden] = LOWEST, LOWEST
    got = run(q, k, v, g)
    want = R.attention(q, k[:, ~hidden], v[:, ~hidden], dout=g)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), got):
        if name in ("dk", "dv"):
            assert torch.count_nonzero(t[:, hidden]) == 0, name
            t = t[:, ~hidden]
        R.check(t, *want[name], name)
