"""GPU parity of layer norm and its gradient against the plain 64-bit form, within bounds
derived from the arithmetic (ops_ref): row and channels-first forms, the three types, f32
parameters, odd sizes, one channel, one row, no rows, unaligned buffers, streams."""
import pytest
import torch

import ops_ref as R
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    yield
    _ops.check_device()


# (shape, axis)
SHAPES = [
    ((7, 768), -1), ((3, 5, 64), -1), ((1, 1), -1), ((1, 8), -1), ((33, 1), -1), ((129, 100), -1),
    ((5, 1001), -1), ((300, 32), -1), ((4, 1024), -1), ((3, 2050), -1), ((2, 4096), -1),
    ((2, 5000), -1), ((3, 8192), -1), ((2, 9001), -1), ((2, 20000), -1), ((1000, 96), -1),
    ((2, 128, 7, 8), 1), ((3, 24, 5), 1), ((2, 96, 14, 14), 1), ((1, 33, 49), 1), ((4, 1, 9), 1),
    ((2, 768, 10), 1), ((1, 2000, 3), 1), ((5, 16, 64), 1), ((3, 40, 2), 1), ((2, 7, 6, 33), 2),
    ((70, 8, 130), 1),
]


def case(shape, axis, dtype, params, seed=5):
    T, P = R.TYPES[dtype], R.TYPES[params]
    C = shape[axis]
    x = R.normal(seed, shape, T, 1.5, 0.4)
    w = R.normal(seed + 1, (C,), P, 0.3, 1.0)
    b = R.normal(seed + 2, (C,), P, 0.2)
    dy = R.normal(seed + 3, shape, T)
    return x, w, b, dy


@pytest.mark.parametrize("dtype,params", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32"),
                                          ("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape,axis", SHAPES)
def test_forward_and_backward(shape, axis, dtype, params):
    x, w, b, dy = case(shape, axis, dtype, params)
    eps = 1e-5
    y, mean, rstd = fc.layer_norm(x.cuda(), w.cuda(), b.cuda(), axis=axis, eps=eps,
                                  return_stats=True)
    ref, m, r, tol = R.layer_norm(x, w, b, axis, eps)
    R.check(y, ref, tol, "y")
    xd = x.double().movedim(axis, -1)
    e = R.norm_error(xd, r)
    R.check(mean, m, e / r, "mean")
    R.check(rstd, r, 2 * e * r + 4 * R.E32 * r, "rstd")
    got = fc.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda(), b.cuda(), axis=axis)
    want = R.layer_norm_backward(dy, x, w, b, axis, eps)
    for name, g in zip(("dx", "dweight", "dbias"), got):
        R.check(g, *want[name], name)


def test_without_parameters_and_inference():
    x, _, _, dy = case((9, 200), -1, "f16", "f16")
    y = fc.layer_norm(x.cuda(), axis=-1, eps=1e-6)
    ref, _, _, tol = R.layer_norm(x, None, None, -1, 1e-6)
    R.check(y, ref, tol, "y")
    y, mean, rstd = fc.layer_norm(x.cuda(), return_stats=True)
    dx, dw, db = fc.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd)
    assert dw is None and db is None
    R.check(dx, *R.layer_norm_backward(dy, x, None, None, -1, 1e-5)["dx"], "dx")
    x, w, b, dy = case((4, 48, 6), 1, "f32", "f32")
    y, mean, rstd = fc.layer_norm(x.cuda(), w.cuda(), axis=1, return_stats=True)
    dx, dw, db = fc.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda(), axis=1)
    want = R.layer_norm_backward(dy, x, w, None, 1, 1e-5)
    assert db is None
    R.check(dx, *want["dx"], "dx")
    R.check(dw, *want["dweight"], "dweight")
    dx2, dw, db = fc.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda(), axis=1,
                                         param_grads=False)
    assert dw is None and db is None and torch.equal(dx, dx2)


def test_far_mean_keeps_the_variance():
    """A mean 4096 deviations away: a one-pass sum of squares would lose the variance."""
    x = R.normal(3, (6, 1536), torch.float32, 1.0, 4096.0)
    w = torch.ones(1536)
    y = fc.layer_norm(x.cuda(), w.cuda(), eps=1e-5)
    ref, _, _, tol = R.layer_norm(x, w, None, -1, 1e-5)
    R.check(y, ref, tol, "y")
    assert float(tol.max()) < 0.2


def test_constant_rows_and_nonfinite_rows():
    x = torch.full((3, 64), 2.5)
    x[1, 5] = float("nan")
    y = fc.layer_norm(x.cuda(), eps=1e-5).cpu()
    assert torch.equal(y[0], torch.zeros(64)) and torch.equal(y[2], torch.zeros(64))
    assert torch.isnan(y[1]).all()


def test_no_rows():
    w = torch.ones(16, device="cuda", dtype=torch.float16)
    x = torch.empty((0, 16), device="cuda", dtype=torch.float16)
    y, mean, rstd = fc.layer_norm(x, w, w, return_stats=True)
    assert y.shape == (0, 16) and mean.shape == (0,)
    dx, dw, db = fc.layer_norm_backward(x, x, mean, rstd, w, w)
    assert dx.shape == (0, 16)
    assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


@pytest.mark.parametrize("shape,axis", [((37, 256), -1), ((3, 24, 40), 1)])
def test_unaligned_buffers_and_guards(shape, axis):
    """Buffers that start one element off a 16-byte boundary give the same values, and nothing
    is written around the output."""
    x, w, b, dy = case(shape, axis, "f16", "f16")
    n = x.numel()

    def off(t):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.cuda().view(-1)
        return buf[1:].view(t.shape)

    buf = torch.full((n + 2 * GUARD + 1,), 7.0, dtype=torch.float16, device="cuda")
    out = buf[GUARD + 1:GUARD + 1 + n].view(shape)
    y, mean, rstd = fc.layer_norm(off(x), off(w), off(b), axis=axis, out=out, return_stats=True)
    ref, _, _, tol = R.layer_norm(x, w, b, axis, 1e-5)
    R.check(y, ref, tol, "y")
    assert (buf[:GUARD + 1] == 7).all() and (buf[GUARD + 1 + n:] == 7).all()
    got = fc.layer_norm_backward(off(dy), off(x), mean, rstd, off(w), off(b), axis=axis)
    want = R.layer_norm_backward(dy, x, w, b, axis, 1e-5)
    for name, g in zip(("dx", "dweight", "dbias"), got):
        R.check(g, *want[name], name)


@pytest.mark.parametrize("shape,axis", [((50, 512), -1), ((2, 64, 36), 1)])
def test_in_place_streams_and_repeats(shape, axis):
    x, w, b, dy = (t.cuda() for t in case(shape, axis, "bf16", "bf16"))
    y, mean, rstd = fc.layer_norm(x, w, b, axis=axis, return_stats=True)
    grads = fc.layer_norm_backward(dy, x, mean, rstd, w, b, axis=axis)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, mean2, rstd2 = fc.layer_norm(x, w, b, axis=axis, return_stats=True, stream=side)
    again = fc.layer_norm_backward(dy, x, mean2, rstd2, w, b, axis=axis, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)
    for a, c in zip(grads, again):
        assert torch.equal(a, c)
    z = x.clone()
    assert fc.layer_norm(z, w, b, axis=axis, out=z) is z and torch.equal(z, y)


def test_gradient_against_differences():
    """Directional differences of the 64-bit loss, within the gradient's own bounds."""
    for shape, axis in [((6, 40), -1), ((2, 24, 9), 1)]:
        x, w, b, dy = case(shape, axis, "f32", "f32")
        _, mean, rstd = fc.layer_norm(x.cuda(), w.cuda(), b.cuda(), axis=axis, return_stats=True)
        got = fc.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda(), b.cuda(), axis=axis)
        want = R.layer_norm_backward(dy, x, w, b, axis, 1e-5)
        loss = lambda x, w, b: (R.layer_norm(x, w, b, axis, 1e-5)[0] * dy.double()).sum()  # noqa
        args = {"dx": x, "dweight": w, "dbias": b}
        R.U[torch.float64], R.TINY[torch.float64] = 2.0 ** -53, 0.0
        for i, (name, t) in enumerate(args.items()):
            d = R.normal(90 + i, t.shape, torch.float64)
            vals = []
            for sign in (1, -1):
                moved = [a.double() for a in args.values()]
                moved[i] = moved[i] + sign * 1e-4 * d
                vals.append(loss(*moved))
            slope = (vals[0] - vals[1]) / 2e-4
            dot = (got[i].double().cpu() * d).sum()
            assert abs(dot - slope) <= (want[name][1] * d.abs()).sum() + 1e-5 * abs(slope) + 1e-6


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are right."""
    C = 2048
    rows = (1 << 31) // C + 5
    x = torch.zeros((rows, C), dtype=torch.float16, device="cuda")
    tail = R.normal(8, (4, C), torch.float16)
    x[-4:] = tail.cuda()
    y, mean, rstd = fc.layer_norm(x, return_stats=True)
    ref, _, _, tol = R.layer_norm(tail, None, None, -1, 1e-5)
    R.check(y[-4:], ref, tol, "y")
    assert torch.count_nonzero(y[:3]) == 0
    del y
    dy = x
    dx, _, _ = fc.layer_norm_backward(dy, x, mean, rstd)
    R.check(dx[-4:], *R.layer_norm_backward(tail, tail, None, None, -1, 1e-5)["dx"], "dx")


def test_inputs_given_back_before_a_side_stream_runs():
    """A call on another stream than its input's: the input may be dropped while the work still
    waits there, and what takes the memory next does not reach the result."""
    x = R.normal(31, (512, 1024), torch.float32).cuda()
    want = fc.layer_norm(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = fc.layer_norm(x, stream=side)
    del x
    again = [torch.full((512, 1024), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(again) == 4
