"""Activations and slopes of the gated block at each gate value, relative to the values themselves:
one hidden unit a gate value, so that nothing else adds to an output and a saturated gate cannot
hide behind others. Bounds from the functions' conditions and roundings."""
import math

import pytest
import torch

import ops_ref as R
from ops_ref import E32, TINY, U
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu

F = 320  # hidden units, a gate value each


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    yield
    _ops.check_device()


def act(kind, v, alpha):
    """(a, the two terms of its slope, size of the exponential's argument) in 64 bits, none of
    them from a difference of close numbers."""
    if kind == "Sigmoid":
        p, q = torch.sigmoid(v), torch.sigmoid(-v)
        return p, p * q, torch.zeros_like(v), v.abs()
    if kind == "Gelu":
        p = 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
        return v * p, p, v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi), 0.5 * v * v
    if kind == "FastGelu":  # (1 + tanh z) / 2 is the logistic function of 2 z
        k = math.sqrt(8.0 / math.pi)
        w, dw = k * (v + 0.044715 * v ** 3), k * (1.0 + 3 * 0.044715 * v * v)
    else:
        w, dw = alpha * v, torch.full_like(v, alpha)
    p, q = torch.sigmoid(w), torch.sigmoid(-w)
    return v * p, p, v * p * q * dw, w.abs()


def off(size):
    """Bound on the relative error of a value that holds exp of an argument of this size: the
    argument is off by at most six roundings (constants, products, the change to base 2), erfc of z
    by z^2 of them twice; the functions, reciprocals and products after them count 32 units (erfcf 4
    ulp, expf 2, division 2, each twice the unit). The 16-bit tensor route's Gelu adds its
    approximation's 3.7e-6, under 64 units."""
    return (8 * size + 96) * E32


def block(values, T, n, route, kind, params):
    """Both passes with gate j at values[j] for every token and up projection scale[j], where the
    incoming gradient of the last token is `dy`; identity as the down projection."""
    a = act(kind, values.double(), params[0] if params else 1.0)[0].abs()
    top = 15 if T == torch.float16 else 90
    scale = 2.0 ** torch.nan_to_num(-a.log2().round(), posinf=0.0).clamp(-14 if top == 15 else -90,
                                                                        top)
    scale = scale.to(T)  # a power of two: h is about 1 where the type has room
    x, g, u = torch.zeros(n, 8, dtype=T), torch.zeros(F, 8, dtype=T), torch.zeros(F, 8, dtype=T)
    x[:, 0], g[:, 0], u[:, 0] = 1.0, values, scale
    dev = [t.cuda() for t in (x, g, u, torch.eye(F).to(T))]
    how = dict(activation=kind, activation_params=params, route=route)
    zero = torch.zeros(F, dtype=T).cuda()
    y, saved = fc.gated_mlp(*dev, b_gate=zero, b_up=zero, **how, return_saved=True)

    def back(row):
        dy = torch.zeros(n, F, dtype=T)
        dy[-1] = row
        return fc.gated_mlp_backward(dy.cuda(), *dev, saved, b_gate=zero, b_up=zero, **how)

    return scale, y, back


KINDS = [("Silu", None), ("QuickGelu", [1.702]), ("Sigmoid", None), ("Gelu", None),
         ("FastGelu", None)]


@pytest.mark.parametrize("route", ["auto", "simple"])
@pytest.mark.parametrize("n", [1, 33, 300])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,params", KINDS)
def test_each_gate_value_relative_to_itself(kind, params, dtype, n, route):
    T = R.TYPES[dtype]
    values = torch.linspace(-8.0, 8.0, F, dtype=torch.float64).add_(0.0137).to(T)
    scale, y, back = block(values, T, n, route, kind, params)
    v, s = values.double(), scale.double()
    a, s1, s2, size = act(kind, v, params[0] if params else 1.0)
    # of a value that one product of each operand's parts carries on: its roundings to T (h, dg and
    # du, and the output), and what three planes or two TF32 parts leave out of it
    rounds = (2.02 * U[T] if T != torch.float32 else 0.0) + 16 * E32
    rel = off(size) + rounds
    h = a * s
    R.check(y, h.expand(n, F), (rel * h.abs() + 2 * TINY[T]).expand(n, F), "y")

    one = back(torch.ones(F, dtype=T))
    dg = s * (s1 + s2)
    tol = off(size) * s * (s1.abs() + s2.abs()) + rounds * dg.abs() + 2 * TINY[T]
    dg_in = dg.abs() < torch.finfo(T).max
    for name, got in (("dw_gate", one[1][:, 0]), ("db_gate", one[4])):
        R.check(got[dg_in.cuda()], dg[dg_in], tol[dg_in], name)
    R.check(one[3].diagonal(), h, rel * h.abs() + 2 * TINY[T], "dw_down")
    scaled = back(scale)
    for name, got in (("dw_up", scaled[2][:, 0]), ("db_up", scaled[5])):
        R.check(got, h, rel * h.abs() + 2 * TINY[T], name)


@pytest.mark.parametrize("route", ["auto", "simple"])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["Silu", "Gelu", "FastGelu", "Sigmoid"])
def test_gates_of_any_size(kind, dtype, n, route):
    """Gates whose square or cube no f32 holds: act(g) is g or 0 (Sigmoid 1 or 0), its slope 1 or 0
    (Sigmoid 0)."""
    T = R.TYPES[dtype]
    values = torch.cat([torch.logspace(2, 38, F // 2), -torch.logspace(2, 38, F // 2)]).to(T)
    x, g, u = torch.zeros(n, 8, dtype=T), torch.zeros(F, 8, dtype=T), torch.zeros(F, 8, dtype=T)
    x[:, 0], g[:, 0], u[:, 0] = 1.0, values, 1.0
    # half an identity: sums hold no more than one value, and none of them passes the type
    dev = [t.cuda() for t in (x, g, u, (torch.eye(F) / 2).to(T))]
    y, saved = fc.gated_mlp(*dev, activation=kind, route=route, return_saved=True)
    dy = torch.zeros(n, F, dtype=T)
    dy[-1] = 2.0
    grads = fc.gated_mlp_backward(dy.cuda(), *dev, saved, activation=kind, route=route)
    v = values.double()
    on = (v > 0).double()
    a = on if kind == "Sigmoid" else v.clamp(min=0.0)
    slope = torch.zeros_like(v) if kind == "Sigmoid" else on
    # at -100 all but Sigmoid's and Silu's exponentials are 0 in f32, and those are under 4e-42
    tiny, rel = 1e-40, 2.02 * U[T] + 32 * E32
    R.check(y[-1], a / 2, rel * a + tiny, "y")
    R.check(grads[2][:, 0], a, rel * a + tiny, "dw_up")
    R.check(grads[1][:, 0], slope, rel * slope + tiny, "dw_gate")
