"""f32 in the gated block keeps its bits through every product: all operands are diagonal powers of
two but one, whose 24-bit values then have to come out as they are; and many tiles a block, results
by boxes and by rows in one launch, and any subset of gradients within derived bounds."""
import pytest
import torch

import block_ref as B
import ops_ref as R
from ops_ref import E32
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops
from test_gpu_mlp import NAMES, both_passes, case, check_all

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    _ops._start()
    yield
    _ops.check_device()


@pytest.mark.parametrize("route", ["auto", "simple"])
@pytest.mark.parametrize("m", [20, 96, 600])
@pytest.mark.parametrize("full", ["x", "gate", "up", "down", "dy"])
def test_every_product_keeps_f32(full, m, route):
    """No activation. A product of a value and a power of two is exact in each of its parts, and
    the parts' sum is cut or rounded a few times at most (three planes, or two TF32 parts the
    second of which is read without its last bits: under 2^-22 of the value a product, so 4 units;
    three products in a row at most, two of them where an output squares the value)."""
    g = torch.Generator().manual_seed(m)
    diag = {k: torch.diag(2.0 ** torch.randint(-3, 4, (m,), generator=g).float())
            for k in ("x", "gate", "up", "down", "dy")}
    diag[full] = torch.diag(1.0 + torch.rand(m, generator=g))
    x, wg, wu, wd, dy = (diag[k] for k in ("x", "gate", "up", "down", "dy"))
    got = both_passes(x, wg, wu, wd, [None] * 3, dy, activation=None, route=route)
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    gp, up = x * wg, x * wu
    h, dh = gp * up, dy * wd
    ref = {"y": h * wd, "dx": dh * up * wg + dh * gp * wu, "dw_gate": dh * up * x,
           "dw_up": dh * gp * x, "dw_down": dy * h}
    for name, val in ref.items():
        R.check(got[name], val, 24 * E32 * val.abs(), name)


@pytest.mark.parametrize("n,c,f,o,activation", [(2600, 520, 1100, 530, "Gelu"),
                                                (1500, 1300, 1700, 90, "FastGelu")])
def test_many_tiles_in_f32(n, c, f, o, activation):
    """Several tiles a block in every product: accumulators, slots and problems change hands."""
    ins = case(300, n, c, f, o, torch.float32)
    check_all(both_passes(*ins, activation=activation), *ins, activation=activation)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,c,f,o,activation", [
    (2600, 1031, 1104, 1048, "FastGelu"),  # dx, dw_gate and dw_up by rows, dw_down by boxes
    (2600, 1032, 1101, 1048, "Gelu"),      # the other way round
    (2440, 1032, 1104, 1047, "Relu"),      # y by rows
])
def test_boxes_and_rows_in_one_launch(n, c, f, o, activation, dtype):
    ins = case(310, n, c, f, o, R.TYPES[dtype])
    check_all(both_passes(*ins, activation=activation), *ins, activation=activation)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,c,f,o", [(40, 96, 136, 64), (300, 96, 136, 64), (700, 520, 640, 264)])
def test_subsets_of_gradients(n, c, f, o, dtype):
    """Launches of fewer products may take other shapes: each within the bounds of the whole call."""
    x, wg, wu, wd, b, dy = case(320, n, c, f, o, R.TYPES[dtype])
    ref = B.gated_mlp(x, wg, wu, wd, *b, dy=dy)
    dev = [t.contiguous().cuda() for t in (dy, x, wg, wu, wd, b[0], b[1])]
    p = fc.MlpPlan(_ops._code(x.dtype), n, c, f, o, x_stride=c, y_stride=o, gate_stride=c,
                   up_stride=c, down_stride=f, dy_stride=o, dx_stride=c, has_b_gate=True,
                   has_b_up=True, has_b_down=True, alpha=1.0, training=True)
    ws = torch.empty(p.backward_workspace, dtype=torch.uint8, device="cuda")
    shapes = [(n, c), (f, c), (f, c), (o, f), (f,), (f,), (o,)]
    for which in ((0,), (1,), (2,), (3,), (4,), (5,), (6,), (0, 1), (2, 3), (1, 2, 3), (0, 4, 5, 6),
                  (3, 6), (0, 3), ()):
        outs = [torch.full(s, float("nan"), dtype=x.dtype, device="cuda") if i in which else None
                for i, s in enumerate(shapes)]
        p.backward_ptrs(*(t.data_ptr() for t in dev), None, *map(_ops._ptr, outs), ws.data_ptr(),
                        ws.numel(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for i in which:
            R.check(outs[i], *ref[NAMES[i]], f"{NAMES[i]} of {which}")
