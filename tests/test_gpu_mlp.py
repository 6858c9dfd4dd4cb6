"""GPU parity of the gated feed-forward block, forward and backward, against the plain 64-bit
form, within bounds derived from the arithmetic (block_ref)."""
import pytest
import torch

import block_ref as B
import ops_ref as R
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dw_gate", "dw_up", "dw_down", "db_gate", "db_up", "db_down")


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    yield
    _ops.check_device()


def case(seed, n, c, f, o, T, biases=True):
    """x, packed gate and up, down, biases and dy."""
    x, dy = R.normal(seed, (n, c), T), R.normal(seed + 1, (n, o), T)
    both = R.normal(seed + 2, (2 * f, c), T, c ** -0.5)
    down = R.normal(seed + 3, (o, f), T, f ** -0.5)
    b = [R.normal(seed + 4 + i, (m,), T, 0.3) for i, m in enumerate((f, f, o))] if biases \
        else [None] * 3
    return x, both[:f], both[f:], down, b, dy


def both_passes(x, wg, wu, wd, b, dy, activation="Silu", params=None, route="auto", saved=True):
    dev = [t.cuda() for t in (x, wg, wu, wd)]
    how = dict(b_gate=b[0], b_up=b[1], b_down=b[2], activation=activation,
               activation_params=params, route=route)
    for k in ("b_gate", "b_up", "b_down"):
        how[k] = None if how[k] is None else how[k].cuda()
    y, kept = fc.gated_mlp(*dev, **how, return_saved=True)
    plain = fc.gated_mlp(*dev, **how)
    assert torch.equal(y, plain)
    grads = fc.gated_mlp_backward(dy.cuda(), *dev, kept if saved else None, **how)
    return {"y": y, **dict(zip(NAMES, grads))}


def check_all(got, x, wg, wu, wd, b, dy, activation="Silu", alpha=1.702):
    ref = B.gated_mlp(x, wg, wu, wd, *b, activation, alpha, dy)
    for name, (val, tol) in ref.items():
        R.check(got[name], val, tol, name)
    for name in NAMES:
        assert name in ref or got[name] is None


SIZES = [
    # tokens, features, hidden, out_features
    (1, 8, 8, 8), (1, 64, 128, 64), (3, 72, 40, 24), (8, 256, 512, 256), (9, 64, 136, 72),
    (17, 96, 200, 104), (33, 128, 64, 128), (100, 200, 264, 136), (128, 64, 128, 256),
    (129, 136, 328, 64), (257, 320, 128, 520), (300, 64, 72, 64),
    # sizes that no 16-byte row has
    (1, 1, 1, 1), (5, 33, 17, 9), (70, 37, 131, 61), (130, 65, 129, 67),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,f,o", SIZES)
def test_forward_and_backward(n, c, f, o, dtype):
    ins = case(10, n, c, f, o, R.TYPES[dtype], biases=(n + f) % 2 == 0)
    check_all(both_passes(*ins), *ins)


@pytest.mark.parametrize("dtype,n", [("f16", 2600), ("bf16", 2440)])
def test_many_tiles(dtype, n):
    """Enough tiles for the variants that fill the GPU, with ragged ends in every axis; the last
    rows leave half of a 256-row tile empty, or part of it."""
    ins = case(15, n, 1032, 1104, 1048, R.TYPES[dtype])
    check_all(both_passes(*ins), *ins)


@pytest.mark.parametrize("route", ["simple", "auto"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("activation,params", [
    ("Silu", None), ("Gelu", None), ("FastGelu", None), ("QuickGelu", None), ("QuickGelu", [0.7]),
    ("Relu", None), ("Sigmoid", None), (None, None)])
@pytest.mark.parametrize("n", [5, 150])
def test_activations(activation, params, dtype, route, n):
    ins = case(20, n, 64, 136, 72, R.TYPES[dtype])
    got = both_passes(*ins, activation=activation, params=params, route=route)
    check_all(got, *ins, activation=activation, alpha=params[0] if params else 1.702)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [4, 140])
def test_projections_made_again_give_the_same_bits(dtype, n):
    ins = case(30, n, 96, 160, 64, R.TYPES[dtype])
    a, b = both_passes(*ins), both_passes(*ins, saved=False)
    for name in a:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("n", [6, 150])
@pytest.mark.parametrize("which", [(0,), (1,), (2,), (0, 2)])
def test_some_biases(n, which):
    x, wg, wu, wd, b, dy = case(40, n, 64, 72, 64, torch.float16)
    b = [t if i in which else None for i, t in enumerate(b)]
    check_all(both_passes(x, wg, wu, wd, b, dy), x, wg, wu, wd, b, dy)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3, 200])
def test_large_projections(dtype, n):
    """Gates far from zero, where the activations and their slopes saturate."""
    x, wg, wu, wd, b, dy = case(50, n, 64, 64, 64, R.TYPES[dtype])
    wg = wg * 16
    for activation in ("Silu", "Gelu", "FastGelu", "Sigmoid"):
        got = both_passes(x, wg, wu, wd, b, dy, activation=activation)
        for name, t in got.items():
            assert torch.isfinite(t).all(), (activation, name)
        check_all(got, x, wg, wu, wd, b, dy, activation=activation)


@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("n", [7, 140])
def test_strided_rows_batches_and_guards(n, shift):
    """Rows inside wider buffers at aligned and unaligned starts; outputs leave the rest alone."""
    c, f, o, T = 64, 136, 72, torch.float16
    x, wg, wu, wd, b, dy = case(60, n, c, f, o, T)

    def inside(t, pad):
        buf = torch.full((t.shape[0] * (t.shape[1] + pad) + shift + 3,), 9.0, dtype=T).cuda()
        view = buf[shift:shift + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], -1)
        view = view[:, :t.shape[1]]
        view.copy_(t.cuda())
        return buf, view

    views = [inside(t, 8)[1] for t in (x, wg, wu, wd)]
    how = dict(b_gate=b[0].cuda(), b_up=b[1].cuda(), b_down=b[2].cuda())
    ybuf, y = inside(torch.zeros(n, o), 16)
    dxbuf, dx = inside(torch.zeros(n, c), 24)
    _, saved = fc.gated_mlp(*views, **how, out=y, return_saved=True)
    grads = fc.gated_mlp_backward(inside(dy, 16)[1], *views, saved, **how, dx=dx)
    assert grads[0].data_ptr() == dx.data_ptr()
    check_all({"y": y, **dict(zip(NAMES, grads))}, x, wg, wu, wd, b, dy)
    for buf, view, pad in ((ybuf, y, 16), (dxbuf, dx, 24)):
        rest = torch.ones_like(buf, dtype=torch.bool)
        at = rest[shift:shift + n * (view.shape[1] + pad)].view(n, -1)
        at[:, :view.shape[1]] = False
        assert (buf[rest] == 9.0).all()
    # leading axes
    if n % 2 == 0:
        got = fc.gated_mlp(views[0].unflatten(0, (2, n // 2)), *views[1:], **how)
        assert torch.equal(got.flatten(0, 1), y)


@pytest.mark.parametrize("n", [12, 300])
def test_rows_with_nan_stay_by_themselves(n):
    x, wg, wu, wd, b, dy = case(70, n, 64, 128, 64, torch.bfloat16)
    clean = fc.gated_mlp(x.cuda(), wg.cuda(), wu.cuda(), wd.cuda())
    x[3, 5], x[n - 1, 0] = float("nan"), float("inf")
    got = fc.gated_mlp(x.cuda(), wg.cuda(), wu.cuda(), wd.cuda())
    same = (clean == got).all(-1)
    assert int((~same).sum()) == 2 and not same[3] and not same[n - 1]
    assert torch.isnan(got[3]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_no_tokens(dtype):
    x, wg, wu, wd, b, dy = case(80, 0, 64, 72, 40, R.TYPES[dtype])
    got = both_passes(x, wg, wu, wd, b, dy)
    assert got["y"].shape == (0, 40) and got["dx"].shape == (0, 64)
    for name in NAMES[1:]:
        assert (got[name] == 0).all(), name


def test_only_some_gradients():
    x, wg, wu, wd, b, dy = case(90, 140, 64, 72, 64, torch.bfloat16)
    whole = both_passes(x, wg, wu, wd, [None] * 3, dy)
    dx, *rest = fc.gated_mlp_backward(dy.cuda(), x.cuda(), wg.cuda(), wu.cuda(), wd.cuda(),
                                      param_grads=False)
    assert torch.equal(dx, whole["dx"]) and rest == [None] * 6


@pytest.mark.parametrize("n", [5, 40])
def test_gradients_match_differences(n):
    """Central differences of a 64-bit loss along random directions."""
    ins = case(100, n, 24, 40, 16, torch.float32)
    x, wg, wu, wd, b, dy = ins
    got = both_passes(*ins, activation="Gelu")
    ref = B.gated_mlp(x, wg, wu, wd, *b, "Gelu", dy=dy)

    def loss(vals):
        X, G, UP, D, bg, bu, bd = vals
        h = B.act("Gelu", X @ G.t() + bg)[0] * (X @ UP.t() + bu)
        return ((h @ D.t() + bd) * dy.double()).sum()

    at = [t.double() for t in (x, wg, wu, wd, *b)]
    for seed in range(3):
        d = [R.normal(200 + 10 * seed + i, t.shape, torch.float64, t.std().item())
             for i, t in enumerate(at)]
        t = 1e-4
        slope = (loss([a + t * e for a, e in zip(at, d)])
                 - loss([a - t * e for a, e in zip(at, d)])) / (2 * t)
        total = sum((got[m].double().cpu() * e).sum() for m, e in zip(NAMES, d))
        tol = sum((ref[m][1] * e.abs()).sum() for m, e in zip(NAMES, d))
        assert abs(total - slope) <= tol + 1e-5 * abs(slope) + 1e-5


@pytest.mark.parametrize("n", [8, 400])
def test_streams_and_a_captured_graph(n):
    """On another stream, and captured twice into one graph with results that repeat bit by bit."""
    x, wg, wu, wd, b, dy = case(110, n, 256, 640, 256, torch.bfloat16)
    dev = [t.cuda() for t in (x, wg, wu, wd)]
    how = dict(b_gate=b[0].cuda(), b_up=b[1].cuda(), b_down=b[2].cuda())
    g = dy.cuda()

    def both(stream=None):
        y, saved = fc.gated_mlp(*dev, **how, return_saved=True, stream=stream)
        return (y, *fc.gated_mlp_backward(g, *dev, saved, **how, stream=stream))

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
        for p, q in zip(got, want):
            assert torch.equal(p, q)


def test_broadcast_rows_of_x():
    x, wg, wu, wd, b, dy = case(120, 1, 64, 72, 64, torch.float16)
    wide = x.cuda().expand(150, 64)
    got = fc.gated_mlp(wide, wg.cuda(), wu.cuda(), wd.cuda())
    val, tol = B.gated_mlp(x.expand(150, 64), wg, wu, wd)["y"]
    R.check(got, val, tol, "y")


def test_offsets_past_32_bits():
    """Rows so far apart that the last ones lie past 2^31 elements."""
    n, c, f = 40, 64, 72
    x, wg, wu, wd, b, dy = case(130, n, c, f, c, torch.bfloat16)
    step = (1 << 31) // 32
    buf = torch.empty(step * (n - 1) + c, dtype=torch.bfloat16, device="cuda")
    wide = buf.as_strided((n, c), (step, 1))
    wide.copy_(x.cuda())
    val, tol = B.gated_mlp(x, wg, wu, wd)["y"]
    for route in ("auto", "simple"):
        got = fc.gated_mlp(wide, wg.cuda(), wu.cuda(), wd.cuda(), route=route)
        R.check(got, val, tol, route)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,f", [(1, 256, 640), (12, 264, 328), (3, 33, 47), (40, 96, 200)])
def test_passes_that_follow_each_other(n, c, f, dtype):
    """Inputs and weights are written in place right before each pass, and passes are not waited
    for: kernels that start beside the ones before them read what those wrote."""
    T = R.TYPES[dtype]
    sets = []
    for i in range(3):
        x, wg, wu, wd, b, dy = case(140 + 10 * i, n, c, f, c, T)
        sets.append([t.cuda() for t in (x, wg, wu, wd, *b, dy)])

    def run(x, wg, wu, wd, bg, bu, bd, dy):
        how = dict(b_gate=bg, b_up=bu, b_down=bd)
        y, saved = fc.gated_mlp(x, wg, wu, wd, **how, return_saved=True)
        return (y, *fc.gated_mlp_backward(dy, x, wg, wu, wd, saved, **how))

    want = []
    for s in sets:
        want.append(run(*s))
        torch.cuda.synchronize()
    buffers = [t.clone() for t in sets[0]]
    got = []
    for i in range(30):
        for b, t in zip(buffers, sets[i % 3]):
            b.copy_(t)
        got.append(run(*buffers))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(outs, want[i % 3]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("n", [16, 32, 33])
def test_two_streams_at_once(n):
    """Calls of two streams, each with a workspace of its own, beside each other."""
    ins = [case(170 + 10 * i, n, 320, 648, 320, torch.bfloat16) for i in range(2)]
    dev = [[t.cuda() for t in (*v[:4], v[5])] for v in ins]

    def run(x, wg, wu, wd, dy):
        y, saved = fc.gated_mlp(x, wg, wu, wd, return_saved=True)
        return (y, *fc.gated_mlp_backward(dy, x, wg, wu, wd, saved)[:4])

    want = [run(*d) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*dev[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for a, b in zip(outs, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("n", [40, 700])
def test_unaligned_rows_in_16_bits(n):
    """Odd sizes and odd strides, which are copied first, and results at odd strides."""
    c, f, o, T = 77, 131, 59, torch.bfloat16
    x, wg, wu, wd, b, dy = case(180, n, c, f, o, T)
    wide = [torch.full((t.shape[0], t.shape[1] + 5), 9.0, dtype=T).cuda() for t in (x, wg, wu, wd, dy)]
    views = []
    for t, w in zip((x, wg, wu, wd, dy), wide):
        w[:, 2:2 + t.shape[1]] = t.cuda()
        views.append(w[:, 2:2 + t.shape[1]])
    how = dict(b_gate=b[0].cuda(), b_up=b[1].cuda(), b_down=b[2].cuda())
    ybuf, dxbuf = torch.full((n, o + 3), 9.0, dtype=T).cuda(), torch.full((n, c + 1), 9.0, dtype=T).cuda()
    y, saved = fc.gated_mlp(*views[:4], **how, return_saved=True, out=ybuf[:, 1:1 + o])
    grads = fc.gated_mlp_backward(views[4], *views[:4], saved, **how, dx=dxbuf[:, :c])
    check_all({"y": y, **dict(zip(NAMES, grads))}, x, wg, wu, wd, b, dy)
    assert (ybuf[:, 0] == 9).all() and (ybuf[:, 1 + o:] == 9).all() and (dxbuf[:, c:] == 9).all()


@pytest.mark.parametrize("n,c,f,o", [(700, 1030, 500, 300), (60, 2000, 130, 90), (150, 90, 1500, 80)])
def test_long_sums_in_f32(n, c, f, o):
    """Sums that are split over passes and over blocks, of every product."""
    ins = case(190, n, c, f, o, torch.float32)
    check_all(both_passes(*ins, activation="Gelu"), *ins, activation="Gelu")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [7, 140])
def test_odd_sizes_in_aligned_rows(n, dtype):
    """Rows that start on 16 bytes but do not fill them are read and written where they are."""
    c, f, o, T = 77, 131, 59, R.TYPES[dtype]
    x, wg, wu, wd, b, dy = case(210, n, c, f, o, T)
    views = []
    for t in (x, wg, wu, wd, dy):
        wide = torch.full((t.shape[0], (t.shape[1] + 15) // 8 * 8), float("nan"), dtype=T).cuda()
        wide[:, :t.shape[1]] = t.cuda()
        views.append(wide[:, :t.shape[1]])
    how = dict(b_gate=b[0].cuda(), b_up=b[1].cuda(), b_down=b[2].cuda())
    ybuf, dxbuf = (torch.full((n, m), 9.0, dtype=T).cuda() for m in (64, 80))
    y, saved = fc.gated_mlp(*views[:4], **how, return_saved=True, out=ybuf[:, :o])
    grads = fc.gated_mlp_backward(views[4], *views[:4], saved, **how, dx=dxbuf[:, :c])
    check_all({"y": y, **dict(zip(NAMES, grads))}, x, wg, wu, wd, b, dy)
    assert (ybuf[:, o:] == 9).all() and (dxbuf[:, c:] == 9).all()


@pytest.mark.parametrize("route", ["simple", "auto"])
@pytest.mark.parametrize("n", [4, 60])
def test_largest_values_in_f32(n, route):
    """Values up to f32's largest, whose first plane would round to an infinity, against weights that
    bring them back."""
    x, wg, wu, wd, b, dy = case(220, n, 64, 72, 40, torch.float32)
    top = torch.finfo(torch.float32).max
    x = (x.double() * 2e38).clamp(-top, top).float()
    x[0, :5] = top
    wg, wu, wd = wg * 1e-33, wu * 1e-33, wd * 1e-9
    b = [t * 1e3 for t in b]
    got = both_passes(x, wg, wu, wd, b, dy, activation="Relu", route=route)
    for name in ("y", "dx", "db_down"):  # the weights' gradients pass the type's largest
        R.check(got[name], *B.gated_mlp(x, wg, wu, wd, *b, "Relu", dy=dy)[name], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [40, 300])
def test_each_gradient_alone(n, dtype):
    """Any subset of the gradients through the plan, with the bits of the whole call."""
    x, wg, wu, wd, b, dy = case(230, n, 96, 136, 64, R.TYPES[dtype])
    whole = both_passes(x, wg, wu, wd, b, dy)
    dev = [t.cuda() for t in (dy, x, wg, wu, wd, b[0], b[1])]
    p = fc.MlpPlan(_ops._code(x.dtype), n, 96, 136, 64, x_stride=96, y_stride=64, gate_stride=96,
                   up_stride=96, down_stride=136, dy_stride=64, dx_stride=96, has_b_gate=True,
                   has_b_up=True, has_b_down=True, training=True)
    ws = torch.empty(p.backward_workspace, dtype=torch.uint8, device="cuda")
    shapes = [(n, 96), (136, 96), (136, 96), (64, 136), (136,), (136,), (64,)]
    for which in ((0,), (1,), (2, 3), (4,), (0, 4, 5, 6), (3, 6), ()):
        outs = [torch.empty(s, dtype=x.dtype, device="cuda") if i in which else None
                for i, s in enumerate(shapes)]
        p.backward_ptrs(*(t.data_ptr() for t in dev), None, *map(_ops._ptr, outs), ws.data_ptr(),
                        ws.numel(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for i in which:
            a, ref = outs[i], whole[NAMES[i]]
            # a launch of fewer products may take another shape, whose sums come in another order
            assert torch.equal(a, ref) or torch.allclose(a.double(), ref.double(), rtol=0.02,
                                                         atol=0.02 * ref.double().abs().max().item())
