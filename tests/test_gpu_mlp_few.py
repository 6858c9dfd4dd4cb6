"""The gated block for up to 32 tokens rounds each 16-bit output once: between its two products
nothing is held in 16 bits, so an output whose terms cancel keeps what they leave."""
import pytest
import torch

import block_ref as B
import ops_ref as R
from ops_ref import U
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops
from test_gpu_mlp import case

pytestmark = pytest.mark.gpu

# What two 16-bit parts leave out of a hidden value: half a step of the second of half a step of
# the first, with as much again for what the second one's own exponent loses.
LEFT = {torch.float16: 2.0 ** -21, torch.bfloat16: 2.0 ** -15}


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    _ops._start()
    yield
    _ops.check_device()


def check(y, x, wg, wu, wd, b, activation):
    T = x.dtype
    f32 = [None if t is None else t.float() for t in (x, wg, wu, wd, *b)]
    ref, tol = B.gated_mlp(*f32, activation)["y"]  # the f32 steps
    X, G, UP, D = (t.double() for t in (x, wg, wu, wd))
    vec = lambda t: 0.0 if t is None else t.double()  # noqa: E731
    h = B.act(activation, X @ G.t() + vec(b[0]))[0] * (X @ UP.t() + vec(b[1]))
    R.check(y, ref, U[T] * ref.abs() * 1.01 + tol + LEFT[T] * (h.abs() @ D.abs().t())
            + R.TINY[T], "y")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("activation", ["Silu", "Gelu"])
@pytest.mark.parametrize("n,c,f,o", [(1, 64, 512, 128), (5, 128, 1000, 72), (8, 64, 40, 16),
                                     (9, 33, 517, 31), (16, 256, 2048, 264), (17, 64, 96, 64),
                                     (32, 200, 776, 136)])
def test_outputs_round_once(n, c, f, o, activation, dtype):
    x, wg, wu, wd, b, _ = case(400, n, c, f, o, R.TYPES[dtype], biases=f % 3 == 1)
    dev = [t.cuda() for t in (x, wg, wu, wd)]
    how = {k: None if t is None else t.cuda() for k, t in zip(("b_gate", "b_up", "b_down"), b)}
    for saved in (False, True):
        y = fc.gated_mlp(*dev, **how, activation=activation, return_saved=saved)
        check(y[0] if saved else y, x, wg, wu, wd, b, activation)


@pytest.mark.parametrize("n", [1, 12, 30])
def test_small_hidden_values_in_f16(n):
    """Hidden values under f16's least normal number, against weights that bring them back."""
    x, wg, wu, wd, b, _ = case(410, n, 64, 264, 40, torch.float16, biases=False)
    x, wd = x / 1024, wd * 64  # h is about 1e-6
    y = fc.gated_mlp(*(t.cuda() for t in (x, wg, wu, wd)))
    check(y * 1.0, x, wg, wu, wd, b, "Silu")


def test_strided_rows():
    n, c, f, o, T = 11, 96, 200, 56, torch.bfloat16
    x, wg, wu, wd, b, _ = case(420, n, c, f, o, T)
    wide = [torch.full((t.shape[0], t.shape[1] + 8), 9.0, dtype=T).cuda() for t in (x, wg, wu, wd)]
    for shift in (0, 1):
        views = []
        for t, w in zip((x, wg, wu, wd), wide):
            w.fill_(9.0)
            w[:, shift:shift + t.shape[1]] = t.cuda()
            views.append(w[:, shift:shift + t.shape[1]])
        out = torch.full((n, o + 5), 9.0, dtype=T).cuda()
        fc.gated_mlp(*views, b_gate=b[0].cuda(), b_up=b[1].cuda(), b_down=b[2].cuda(),
                     out=out[:, 1:1 + o])
        check(out[:, 1:1 + o], x, wg, wu, wd, b, "Silu")
        assert (out[:, 0] == 9).all() and (out[:, 1 + o:] == 9).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,f", [(1, 5), (9, 517), (30, 775), (3, 64)])
def test_what_the_workspace_held_is_not_read(n, f, dtype):
    """A workspace of NaN: rows of hidden values end inside a unit of 16 bytes."""
    c, o, T = 40, 24, R.TYPES[dtype]
    x, wg, wu, wd, b, _ = case(430, n, c, f, o, T)
    dev = [t.contiguous().cuda() for t in (x, wg, wu, wd, *b)]
    p = fc.MlpPlan(_ops._code(T), n, c, f, o, x_stride=c, y_stride=o, gate_stride=c, up_stride=c,
                   down_stride=f, has_b_gate=True, has_b_up=True, has_b_down=True)
    ws = torch.full((p.forward_workspace,), 255, dtype=torch.uint8, device="cuda")
    y = torch.empty((n, o), dtype=T, device="cuda")
    p.forward_ptrs(*(t.data_ptr() for t in dev), y.data_ptr(), None, ws.data_ptr(), ws.numel(),
                   torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    check(y, x, wg, wu, wd, b, "Silu")
