"""Host-side tests of the head norms with rotation and of the gated feed-forward block (no GPU):
structure layouts, refusals of descriptors and of calls, which come before any launch, and the
64-bit forms of the GPU tests against automatic differentiation."""
import ctypes
import os
import subprocess

import pytest
import torch

import block_ref as B
import ops_ref as R
from activation_implicit_gemm_gb300 import FconvError, MlpPlan, NormRopePlan, _build, _ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, F16, BF16 = 0, 1, 2
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    _ops._start()
    return _ops.load()


def code(fn, *a, **kw):
    with pytest.raises(FconvError) as e:
        fn(*a, **kw)
    return e.value.code


def test_struct_layouts_match_the_header(tmp_path):
    checks = [("fconv_norm_rope_desc", _ops.NormRopeDesc),
              ("fconv_mlp_desc", _ops.MlpDesc)]
    body = "".join(f'printf("%zu ", sizeof({c}));' + "".join(
        f'printf("%zu ", offsetof({c}, {f}));' for f, _ in s._fields_) for c, s in checks)
    probe = tmp_path / "probe.c"
    probe.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fconv_ops.h"\n'
                     "int main(void){" + body + "return 0;}\n")
    exe = str(tmp_path / "probe")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(probe), "-o", exe])
    got = [int(v) for v in subprocess.check_output([exe], text=True).split()]
    want = []
    for _, s in checks:
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f, _ in s._fields_]
    assert got == want


# ------------------------------------------------------------------------------ head norms

def heads(dtype=F16, b=2, n=5, hq=4, hk=2, d=16, **kw):
    args = dict(q_stride=(n * hq * d, hq * d, d), q_out_stride=(n * hq * d, hq * d, d),
                k_stride=(n * hk * d, hk * d, d), k_out_stride=(n * hk * d, hk * d, d),
                dq_stride=(n * hq * d, hq * d, d), dk_stride=(n * hk * d, hk * d, d),
                has_k_weight=hk > 0, sections=(4, 4))
    return NormRopePlan(dtype, b, n, hq, hk, d, **{**args, **kw})


def test_norm_rope_refusals():
    assert heads().workspace_bytes == 0
    assert heads(training=True).workspace_bytes >= 16 * 4
    assert code(heads, 7) == "E_UNSUPPORTED"
    assert code(heads, param_dtype=BF16) == "E_UNSUPPORTED"
    heads(param_dtype=F32)
    assert code(heads, d=513) == "E_UNSUPPORTED"
    assert code(heads, hq=65535, hk=1) == "E_UNSUPPORTED"
    assert code(heads, b=1 << 15, n=1 << 12) == "E_UNSUPPORTED"
    assert code(heads, hq=0) == "E_EXTENT"
    assert code(heads, b=-1) == "E_EXTENT"
    assert code(heads, sections=(4, 5)) == "E_EXTENT"
    assert code(heads, pos_batch=3) == "E_EXTENT"
    heads(pos_batch=2)
    heads(sections=())
    for eps in (0.0, -1.0, NAN, INF):
        assert code(heads, eps=eps) == "E_ATTR_VALUE"
    assert code(heads, sections=(4, -1)) == "E_ATTR_VALUE"
    assert code(heads, pos_type=3) == "E_ATTR_VALUE"
    assert code(heads, sections=(1, 1, 1, 1)) == "E_ATTR_VALUE"
    assert code(heads, hk=0, has_k_weight=True) == "E_BIAS_SHAPE"
    assert code(heads, q_stride=(-1, 64, 16)) == "E_STRIDE"
    heads(q_stride=(0, 64, 16))  # an input may be broadcast
    assert code(heads, q_out_stride=(0, 64, 16)) == "E_STRIDE"
    assert code(heads, k_out_stride=(160, 32, 8)) == "E_STRIDE"
    heads(q_out_stride=(0, 64, 16), training=True)  # there it is an input
    assert code(heads, dq_stride=(0, 64, 16), training=True) == "E_STRIDE"
    with pytest.raises(ValueError):
        heads(pairing="pairs")


def test_norm_rope_call_refusals():
    p = heads()
    ok = dict(q=1 << 12, k=2 << 12, w=3 << 12, kw=4 << 12, positions=5 << 12, inv_freq=6 << 12,
              q_out=7 << 12, k_out=8 << 12)

    def run(**kw):
        return code(p.forward_ptrs, *{**ok, **kw}.values(), None)

    for name in ("q", "k", "w", "kw", "positions", "inv_freq", "q_out", "k_out"):
        assert run(**{name: None}) == "E_NULL", name
        assert run(**{name: ok[name] + 1}) == "E_ALIGNMENT", name
    for name in ("k", "w", "kw", "positions", "inv_freq"):
        assert run(q_out=ok[name]) == "E_ALIAS", name
    assert run(k_out=ok["q"]) == "E_ALIAS" and run(k_out=ok["q_out"]) == "E_ALIAS"
    wide = heads(q_out_stride=(5 * 128, 128, 16))
    assert code(wide.forward_ptrs, *{**ok, "q_out": ok["q"]}.values(), None) == "E_ALIAS"
    bare = heads(has_weight=False)
    assert code(bare.forward_ptrs, *ok.values(), None) == "E_BIAS_SHAPE"
    alone = heads(hk=0)
    assert code(alone.forward_ptrs, *{**ok, "kw": None}.values(), None) == "E_EXTENT"
    still = heads(sections=())
    assert code(still.forward_ptrs, *ok.values(), None) == "E_EXTENT"
    heads(b=0).forward_ptrs(None, None, 16, 16, None, None, None, None, None)
    assert code(heads(training=True).forward_ptrs, *ok.values(), None) == "E_UNSUPPORTED"


def test_norm_rope_backward_refusals():
    p = heads(training=True)
    names = ("dq_out", "dk_out", "q", "k", "w", "kw", "positions", "inv_freq", "dq", "dk", "dw",
             "dkw", "ws")
    ok = {n: (i + 1) << 12 for i, n in enumerate(names)}

    def run(plan=p, nbytes=p.workspace_bytes, **kw):
        return code(plan.backward_ptrs, *{**ok, **kw}.values(), nbytes, None)

    for name in names[:10]:
        assert run(**{name: None}) == "E_NULL", name
    for name in names:
        assert run(**{name: ok[name] + 1}) == "E_ALIGNMENT", name
    assert run(ws=None) == "E_WORKSPACE" and run(nbytes=p.workspace_bytes - 1) == "E_WORKSPACE"
    for out in ("dq", "dk", "dw", "dkw"):
        for name in ("q", "k", "w", "kw", "positions", "inv_freq"):
            assert run(**{out: ok[name]}) == "E_ALIAS", (out, name)
    assert run(dq=ok["dk_out"]) == "E_ALIAS" and run(dk=ok["dq_out"]) == "E_ALIAS"
    assert run(dk=ok["dq"]) == "E_ALIAS" and run(dkw=ok["dw"]) == "E_ALIAS"
    assert run(dw=ok["dq_out"]) == "E_ALIAS"
    wide = heads(training=True, dq_stride=(5 * 128, 128, 16))
    assert run(plan=wide, dq=ok["dq_out"]) == "E_ALIAS"
    assert run(plan=heads(training=True, has_weight=False), w=None) == "E_BIAS_SHAPE"
    assert code(heads().backward_ptrs, *ok.values(), 1 << 20, None) == "E_UNSUPPORTED"


def test_norm_rope_arguments(monkeypatch):
    calls = []
    monkeypatch.setattr(_ops, "_run", lambda device, call, *a: calls.append(device))
    monkeypatch.setattr(_ops, "_current_stream", lambda device: 0)

    class Here(torch.Tensor):
        def get_device(self):
            return 1

    def t(*shape, dtype=torch.float16):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Here)

    q, k, w = t(2, 3, 4, 16), t(2, 3, 2, 16), t(16)
    pos, freq = t(3, dtype=torch.int32), t(8, dtype=torch.float32)
    _ops.norm_rope(q, k, weight=w, k_weight=w, positions=pos, inv_freq=freq)
    _ops.norm_rope(q)
    _ops.norm_rope_backward(q, q, k, k, weight=w, positions=pos, inv_freq=freq)
    assert calls == [1, 1, 1]
    bad = [dict(weight=t(15)), dict(weight=t(16), k_weight=t(16, dtype=torch.float32)),
           dict(positions=pos), dict(inv_freq=freq), dict(sections=(8,)),
           dict(positions=t(4, dtype=torch.int32), inv_freq=freq),
           dict(positions=pos, inv_freq=t(7, dtype=torch.float32), sections=(8,)),
           dict(out=t(2, 3, 4, 8)), dict(k_out=t(2, 3, 2, 16, dtype=torch.float32)),
           dict(weight=torch.zeros(16, dtype=torch.float16))]
    for kw in bad:
        with pytest.raises(ValueError):
            _ops.norm_rope(q, k, **kw)
    for a in ((q, t(2, 3, 2, 8)), (q, t(2, 4, 2, 16)), (t(3, 4, 16),),
              (t(2, 3, 16, 4).transpose(2, 3),)):
        with pytest.raises(ValueError):
            _ops.norm_rope(*a)
    with pytest.raises(ValueError, match="k_weight"):
        _ops.norm_rope(q, k_weight=w)
    for kw in (dict(k=k), dict(dk_out=k), dict(dq=t(2, 3, 4, 8))):
        with pytest.raises(ValueError):
            _ops.norm_rope_backward(q, q, **kw)
    assert calls == [1, 1, 1]


# ------------------------------------------------------------------------ feed-forward block

def mlp(dtype=F16, n=10, c=64, f=96, o=32, **kw):
    args = dict(x_stride=c, y_stride=o, gate_stride=c, up_stride=c, down_stride=f, dy_stride=o,
                dx_stride=c, has_b_gate=True, has_b_up=True, has_b_down=True)
    return MlpPlan(dtype, n, c, f, o, **{**args, **kw})


def test_mlp_refusals():
    p = mlp(training=True)
    assert p.forward_workspace >= 10 * 96 * 2 and p.backward_workspace >= 3 * 10 * 96 * 2
    assert p.saved_bytes >= 10 * 96 * 8
    assert code(mlp, 9) == "E_UNSUPPORTED"
    for kw in (dict(n=-1), dict(c=0), dict(f=0), dict(o=0)):
        assert code(mlp, **kw) == "E_EXTENT"
    mlp(n=0)
    for act in (2, 4, 5, 14, 15, -1):
        assert code(mlp, activation=act) == "E_ACTIVATION"
    for alpha in (NAN, INF):
        assert code(mlp, alpha=alpha) == "E_ATTR_VALUE"
    for name in ("x_stride", "gate_stride", "up_stride", "down_stride"):
        assert code(mlp, **{name: -1}) == "E_STRIDE"
    assert code(mlp, y_stride=31) == "E_STRIDE"
    mlp(n=1, y_stride=0)
    assert code(mlp, training=True, dx_stride=63) == "E_STRIDE"
    assert code(mlp, training=True, dy_stride=-8) == "E_STRIDE"
    assert code(mlp, n=1 << 29, f=1 << 20) == "E_UNSUPPORTED"
    for dtype in (F32, F16, BF16):
        assert mlp(dtype).route == "tc" and mlp(dtype, route="simple").route == "simple"


def test_mlp_call_refusals():
    p = mlp()
    names = ("x", "wg", "wu", "wd", "bg", "bu", "bd", "y", "saved", "ws")
    ok = {n: (i + 1) << 12 for i, n in enumerate(names)}

    def run(plan=p, nbytes=1 << 20, **kw):
        return code(plan.forward_ptrs, *{**ok, **kw}.values(), nbytes, None)

    for name in names[:8]:
        assert run(**{name: None}) == "E_NULL", name
    for name in names:
        assert run(**{name: ok[name] + 1}) == "E_ALIGNMENT", name
    for name in names[:7]:
        assert run(y=ok[name]) == "E_ALIAS" and run(saved=ok[name]) == "E_ALIAS", name
    assert run(saved=ok["y"]) == "E_ALIAS"
    assert run(ws=None) == "E_WORKSPACE" and run(nbytes=p.forward_workspace - 1) == "E_WORKSPACE"
    for i, name in enumerate(("has_b_gate", "has_b_up", "has_b_down")):
        assert run(plan=mlp(**{name: False})) == "E_BIAS_SHAPE"
    many = mlp(n=100, route="tc")  # TMA would read x where it is
    assert run(plan=many, x=ok["x"] + 2) == "E_ALIGNMENT"
    empty = dict(ok, x=None, y=None, ws=None)
    mlp(n=0).forward_ptrs(*empty.values(), 0, None)


def test_mlp_backward_refusals():
    p = mlp(training=True)
    names = ("dy", "x", "wg", "wu", "wd", "bg", "bu", "saved", "dx", "dwg", "dwu", "dwd", "dbg",
             "dbu", "dbd", "ws")
    ok = {n: (i + 1) << 12 for i, n in enumerate(names)}

    def run(plan=p, nbytes=1 << 24, **kw):
        return code(plan.backward_ptrs, *{**ok, **kw}.values(), nbytes, None)

    for name in names[:7]:
        assert run(**{name: None}) == "E_NULL", name
    for name in names:
        assert run(**{name: ok[name] + 1}) == "E_ALIGNMENT", name
    for out in names[8:15]:
        for name in names[:8]:
            assert run(**{out: ok[name]}) == "E_ALIAS", (out, name)
    assert run(dwu=ok["dwg"]) == "E_ALIAS"
    n = p.backward_workspace
    assert run(nbytes=n - p.saved_bytes - 1) == "E_WORKSPACE"
    assert run(saved=None, nbytes=n - 1) == "E_WORKSPACE" and run(ws=None) == "E_WORKSPACE"
    assert run(plan=mlp(training=True, has_b_down=False)) == "E_BIAS_SHAPE"
    assert run(plan=mlp()) == "E_UNSUPPORTED"


def test_mlp_arguments(monkeypatch):
    calls = []
    monkeypatch.setattr(_ops, "_run", lambda device, call, *a: calls.append(call.__name__))
    monkeypatch.setattr(_ops, "_current_stream", lambda device: 0)

    class Here(torch.Tensor):
        def get_device(self):
            return 0

    def t(*shape, dtype=torch.float16):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Here)

    x, g, d, b, bd = t(2, 5, 24), t(40, 24), t(16, 40), t(40), t(16)
    for act, params in (("Silu", None), ("QuickGelu", [1.5]), ("Gelu", None), (None, None)):
        y = _ops.gated_mlp(x, g, g, d, b_gate=b, b_up=b, b_down=bd, activation=act,
                           activation_params=params)
        assert y.shape == (2, 5, 16)
    y, saved = (v.as_subclass(Here) for v in _ops.gated_mlp(x, g, g, d, return_saved=True))
    out = _ops.gated_mlp_backward(y, x, g, g, d, saved)
    assert [None if v is None else tuple(v.shape) for v in out] == \
        [(2, 5, 24), (40, 24), (40, 24), (16, 40), None, None, None]
    done = len(calls)
    bad = [(t(24), g, g, d), (x, t(40, 23), g, d), (x, g, t(41, 24), d), (x, g, g, t(16, 41)),
           (x, g, g, t(16, 40, dtype=torch.float32)), (t(2, 24, 5).transpose(1, 2), g, g, d),
           (t(2, 7, 24)[:, 1:6], g, g, d), (x, t(24, 40).t(), g, d), (x, t(1, 40, 24), g, d)]
    for a in bad:
        with pytest.raises(ValueError):
            _ops.gated_mlp(*a)
    for kw in (dict(b_gate=t(39)), dict(b_down=t(40)), dict(b_up=t(40, dtype=torch.float32)),
               dict(activation="Tanh"), dict(activation="Silu", activation_params=[1.0]),
               dict(activation="QuickGelu", activation_params=[1.0, 2.0]),
               dict(activation="Gelu", activation_params=[1.0]), dict(out=t(2, 5, 24)),
               dict(route="fast"), dict(b_up=torch.zeros(40, dtype=torch.float16).float())):
        with pytest.raises(ValueError):
            _ops.gated_mlp(x, g, g, d, **kw)
    for kw in (dict(saved=saved[1:]), dict(saved=t(saved.numel())), dict(dx=t(2, 5, 23))):
        with pytest.raises(ValueError):
            _ops.gated_mlp_backward(y, x, g, g, d, **kw)
    with pytest.raises(ValueError):
        _ops.gated_mlp_backward(t(2, 5, 15), x, g, g, d)
    assert len(calls) == done


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 0)

    class There(torch.Tensor):
        def get_device(self):
            return 1

    q = torch.zeros(1, 2, 2, 8).as_subclass(There)
    w = torch.zeros(8, 8).as_subclass(There)
    for call in (lambda: _ops.norm_rope(q, stream=Stream()),
                 lambda: _ops.norm_rope_backward(q, q, stream=Stream()),
                 lambda: _ops.gated_mlp(w, w, w, w, stream=Stream()),
                 lambda: _ops.gated_mlp_backward(w, w, w, w, w, stream=Stream())):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_plan_caches_drop_their_oldest(monkeypatch):
    monkeypatch.setattr(_ops, "_run", lambda *a: None)
    monkeypatch.setattr(_ops, "_on_cuda", lambda *a: None)
    monkeypatch.setattr(_ops, "_current_stream", lambda device: 0)
    monkeypatch.setattr(_ops, "_KEPT", 4)
    for cache in (_ops._norm_rope_plans, _ops._mlp_plans):
        cache.clear()
    w = torch.zeros(8, 8)
    for n in range(1, 10):
        _ops.norm_rope(torch.zeros(1, n, 2, 8))
        _ops.gated_mlp(torch.zeros(n, 8), w, w, w)
    assert len(_ops._norm_rope_plans) == 4 and len(_ops._mlp_plans) == 4
    for cache in (_ops._norm_rope_plans, _ops._mlp_plans):
        cache.clear()


# --------------------------------------------------------------------------- 64-bit forms

@pytest.mark.parametrize("pairing", ["half", "interleaved", "half_per_axis"])
def test_norm_rope_form_against_autograd(pairing):
    x, dy = R.normal(1, (2, 7, 3, 20), torch.float64), R.normal(2, (2, 7, 3, 20), torch.float64)
    w = R.normal(3, (20,), torch.float64)
    R.U[torch.float64], R.TINY[torch.float64] = 2.0 ** -53, 0.0
    pos = torch.arange(14).view(7, 2)
    freq = torch.rand(8, generator=torch.Generator().manual_seed(4))
    x.requires_grad_(), w.requires_grad_()
    z = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
    y = B._turn(z, pos, freq, (3, 5), pairing)[0]
    y.backward(dy)
    assert torch.allclose(y, B.norm_rope(x.detach(), w.detach(), pos, freq, (3, 5), pairing, 1e-6)[0])
    ref = B.norm_rope_backward(dy, x.detach(), w.detach(), pos, freq, (3, 5), pairing, 1e-6)
    assert torch.allclose(x.grad, ref["dx"][0]) and torch.allclose(w.grad, ref["dw"][0])


@pytest.mark.parametrize("kind", ["Silu", "Gelu", "FastGelu", "QuickGelu", "Relu", "Sigmoid", None])
def test_mlp_form_against_autograd(kind):
    R.U[torch.float64], R.TINY[torch.float64] = 2.0 ** -53, 0.0
    F = torch.nn.functional
    acts = {"Silu": F.silu, "Gelu": F.gelu, "FastGelu": lambda v: F.gelu(v, approximate="tanh"),
            "QuickGelu": lambda v: v * torch.sigmoid(1.702 * v), "Relu": F.relu,
            "Sigmoid": torch.sigmoid, None: lambda v: v}
    x, wg, wu, wd = (R.normal(i, s, torch.float64).requires_grad_()
                     for i, s in enumerate(((9, 6), (11, 6), (11, 6), (5, 11))))
    b = [R.normal(10 + i, (n,), torch.float64).requires_grad_() for i, n in enumerate((11, 11, 5))]
    dy = R.normal(20, (9, 5), torch.float64)
    h = acts[kind](F.linear(x, wg, b[0])) * F.linear(x, wu, b[1])
    y = F.linear(h, wd, b[2])
    y.backward(dy)
    plain = [t.detach() for t in (x, wg, wu, wd, *b)]
    ref = B.gated_mlp(*plain, kind, dy=dy)
    assert torch.allclose(y, ref["y"][0])
    for t, name in zip((x, wg, wu, wd, *b), ("dx", "dw_gate", "dw_up", "dw_down", "db_gate",
                                             "db_up", "db_down")):
        assert torch.allclose(t.grad, ref[name][0]), name
