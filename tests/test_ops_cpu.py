"""Host-side tests of the token-side operators' C ABI (no GPU): exported symbols, structure
layouts, refusals of descriptors and of calls. A call's checks come before any launch, so they
run without a GPU. Also the 64-bit forms that the GPU tests compare with, against PyTorch."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import ops_ref as R
from activation_implicit_gemm_gb300 import (AttentionPlan, FconvError, LayerNormPlan, RopePlan,
                                            _build, _lib, _ops, attention, layer_norm, rope,
                                            rope_frequencies)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _ops.load()


def code(fn, *a, **kw):
    with pytest.raises(FconvError) as e:
        fn(*a, **kw)
    return e.value.code


def test_every_header_function_is_exported_and_declared(lib):
    src = open(os.path.join(ROOT, "include", "fconv_ops.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(fconv_[a-z_]+)\s*\(", src))
    assert len(names) >= 16
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert names <= set(re.findall(r"\sT\s(\w+)$", out, flags=re.M))
    assert names == set(_ops._PROTOS)


def test_struct_layouts_match_the_header(lib, tmp_path):
    checks = [("fconv_norm_desc", _ops.NormDesc, ["channels", "eps"]),
              ("fconv_rope_desc", _ops.RopeDesc, ["q_stride", "axes", "section", "inverse"]),
              ("fconv_attn_desc", _ops.AttnDesc, ["q_stride", "dv_stride", "scale", "training"])]
    body = "".join(f'printf("%zu ", sizeof({c}));' + "".join(
        f'printf("%zu ", offsetof({c}, {f}));' for f in fs) for c, _, fs in checks)
    probe = tmp_path / "probe.c"
    probe.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fconv_ops.h"\n'
                     "int main(void){" + body + "return 0;}\n")
    exe = str(tmp_path / "probe")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(probe), "-o", exe])
    got = [int(v) for v in subprocess.check_output([exe], text=True).split()]
    want = []
    for _, s, fs in checks:
        want += [ctypes.sizeof(s)] + [getattr(s, f).offset for f in fs]
    assert got == want


def test_status_texts(lib):
    for c in _lib.STATUS:
        assert b"unknown status" not in lib.fconv_ops_status_string(c)


def test_norm_refusals(lib):
    ok = LayerNormPlan(BF16, 3, 40, 5, param_dtype=F32)
    assert ok.workspace_bytes >= 2 * 40 * 4
    assert code(LayerNormPlan, 7, 3, 40) == "E_UNSUPPORTED"
    assert code(LayerNormPlan, F16, 3, 40, param_dtype=BF16) == "E_UNSUPPORTED"
    assert code(LayerNormPlan, F16, -1, 40) == "E_EXTENT"
    assert code(LayerNormPlan, F16, 3, 0) == "E_EXTENT"
    assert code(LayerNormPlan, F16, 3, 4, 0) == "E_EXTENT"
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert code(LayerNormPlan, F16, 3, 40, eps=eps) == "E_ATTR_VALUE"
    assert code(LayerNormPlan, F16, 1 << 33, 40) == "E_UNSUPPORTED"


def test_norm_call_refusals(lib):
    p = LayerNormPlan(F16, 3, 40)
    A = 0x10000  # made-up addresses: never read on these paths
    f = lambda **k: code(p.forward_ptrs, *{**dict(x=A, w=2 * A, b=3 * A, y=4 * A, m=5 * A, r=6 * A,  # noqa
                                                 s=None), **k}.values())
    assert f(x=None) == "E_NULL" and f(w=None) == "E_NULL" and f(b=None) == "E_NULL"
    assert f(x=A + 1) == "E_ALIGNMENT" and f(m=5 * A + 2) == "E_ALIGNMENT"
    assert f(y=2 * A) == "E_ALIAS" and f(m=6 * A) == "E_ALIAS"
    g = lambda **k: code(p.backward_ptrs, *{**dict(dy=A, x=2 * A, w=3 * A, m=4 * A, r=5 * A,  # noqa
                                                  dx=6 * A, dw=7 * A, db=8 * A, ws=9 * A,
                                                  n=p.workspace_bytes, s=None), **k}.values())
    assert g(m=None) == "E_NULL" and g(dx=None) == "E_NULL" and g(w=None) == "E_NULL"
    assert g(dx=2 * A) == "E_ALIAS" and g(dw=8 * A) == "E_ALIAS"
    assert g(ws=None) == "E_WORKSPACE" and g(n=p.workspace_bytes - 1) == "E_WORKSPACE"
    q = LayerNormPlan(F16, 3, 40, has_weight=False, has_bias=False)
    assert code(q.forward_ptrs, A, 2 * A, None, 4 * A, None, None, None) == "E_BIAS_SHAPE"
    assert code(q.backward_ptrs, A, 2 * A, None, 4 * A, 5 * A, 6 * A, 7 * A, None, 9 * A, 1 << 20,
                None) == "E_BIAS_SHAPE"


ROPE = dict(q_stride=(640, 64, 16), q_out_stride=(640, 64, 16), k_stride=(320, 32, 16),
            k_out_stride=(320, 32, 16), sections=(3, 5))


def rope_plan(dtype=F16, b=2, t=10, hq=4, hk=2, d=16, **kw):
    return RopePlan(dtype, b, t, hq, hk, d, **{**ROPE, **kw})


def test_rope_refusals(lib):
    rope_plan()
    rope_plan(q_stride=(0, 64, 16))
    assert code(rope_plan, dtype=9) == "E_UNSUPPORTED"
    assert code(rope_plan, hq=0) == "E_EXTENT" and code(rope_plan, d=0) == "E_EXTENT"
    assert code(rope_plan, sections=(4, 5)) == "E_EXTENT"
    assert code(rope_plan, pos_batch=3) == "E_EXTENT"
    assert code(rope_plan, sections=(-1, 5)) == "E_ATTR_VALUE"
    assert code(rope_plan, sections=(1, 1, 1, 1)) == "E_ATTR_VALUE"
    assert code(rope_plan, sections=()) == "E_ATTR_VALUE"
    assert code(rope_plan, pos_type=3) == "E_ATTR_VALUE"
    assert code(rope_plan, q_out_stride=(0, 64, 16)) == "E_STRIDE"
    assert code(rope_plan, q_out_stride=(640, 48, 16)) == "E_STRIDE"
    assert code(rope_plan, k_out_stride=(320, 32, 15)) == "E_STRIDE"
    assert code(rope_plan, q_stride=(640, 64, -16)) == "E_STRIDE"
    with pytest.raises(ValueError):
        rope_plan(pairing="odd")


def test_rope_call_refusals(lib):
    p = rope_plan()
    A = 0x10000
    f = lambda **k: code(p.run_ptrs, *{**dict(q=A, k=2 * A, pos=3 * A, fr=4 * A, qo=5 * A,  # noqa
                                              ko=6 * A, s=None), **k}.values())
    for name in ("q", "k", "pos", "fr", "qo", "ko"):
        assert f(**{name: None}) == "E_NULL"
    assert f(q=A + 1) == "E_ALIGNMENT" and f(pos=3 * A + 2) == "E_ALIGNMENT"
    assert f(qo=2 * A) == "E_ALIAS" and f(ko=5 * A) == "E_ALIAS" and f(ko=A) == "E_ALIAS"
    one = RopePlan(F16, 2, 10, 4, 0, 16, q_stride=(640, 64, 16), q_out_stride=(640, 16, 160),
                   sections=(8,))
    assert code(one.run_ptrs, A, None, 3 * A, 4 * A, A, None, None) == "E_ALIAS"
    assert code(one.run_ptrs, A, 2 * A, 3 * A, 4 * A, 5 * A, None, None) == "E_EXTENT"


def attn_plan(dtype=F16, b=2, lq=5, lk=7, hq=4, hk=2, d=16, **kw):
    s, t = (lq * hq * d, hq * d, d), (lk * hk * d, hk * d, d)
    base = dict(q_stride=s, k_stride=t, v_stride=t, out_stride=s, dout_stride=s, dq_stride=s,
                dk_stride=t, dv_stride=t, training=True)
    return AttentionPlan(dtype, b, lq, lk, hq, hk, d, **{**base, **kw})


def test_attention_refusals(lib):
    attn_plan()
    assert code(attn_plan, dtype=5) == "E_UNSUPPORTED"
    assert code(attn_plan, d=257) == "E_UNSUPPORTED"
    assert code(attn_plan, hq=3) == "E_EXTENT" and code(attn_plan, hk=0) == "E_EXTENT"
    assert code(attn_plan, d=0) == "E_EXTENT" and code(attn_plan, b=-1) == "E_EXTENT"
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert code(attn_plan, scale=scale) == "E_ATTR_VALUE"
    assert code(attn_plan, out_stride=(320, 64, 0)) == "E_STRIDE"
    assert code(attn_plan, dk_stride=(0, 32, 16)) == "E_STRIDE"
    assert code(attn_plan, k_stride=(224, -32, 16)) == "E_STRIDE"
    attn_plan(k_stride=(0, 32, 16), dk_stride=(0, 0, 0), dv_stride=(0, 0, 0), training=False)
    assert code(attn_plan, b=1 << 20, hq=1 << 14) == "E_UNSUPPORTED"


def test_attention_call_refusals(lib):
    p = attn_plan(has_kv_lens=True)
    A = 0x10000
    n = p.forward_workspace
    f = lambda **k: code(p.forward_ptrs, *{**dict(q=A, k=2 * A, v=3 * A, ql=None, kl=4 * A,  # noqa
                                                  o=5 * A, lse=6 * A, ws=7 * A, n=n, s=None),
                                           **k}.values())
    assert f(q=None) == "E_NULL" and f(v=None) == "E_NULL" and f(o=None) == "E_NULL"
    assert f(kl=None) == "E_MASK" and f(ql=8 * A) == "E_MASK"
    assert f(k=2 * A + 1) == "E_ALIGNMENT" and f(lse=6 * A + 2) == "E_ALIGNMENT"
    assert f(o=A) == "E_ALIAS"
    m = p.backward_workspace
    g = lambda **k: code(p.backward_ptrs, *{**dict(do=A, q=2 * A, k=3 * A, v=4 * A, o=5 * A,  # noqa
                                                   lse=6 * A, ql=None, kl=7 * A, dq=8 * A,
                                                   dk=9 * A, dv=10 * A, ws=11 * A, n=m, s=None),
                                            **k}.values())
    assert g(do=None) == "E_NULL" and g(lse=None) == "E_NULL" and g(dv=None) == "E_NULL"
    assert g(dq=A) == "E_ALIAS" and g(dk=8 * A) == "E_ALIAS" and g(dv=3 * A) == "E_ALIAS"
    assert g(kl=None) == "E_MASK"
    assert g(ws=None) == "E_WORKSPACE" and g(n=m - 1) == "E_WORKSPACE"
    once = attn_plan(training=False)
    assert code(once.backward_ptrs, A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, None, None, 8 * A, 9 * A,
                10 * A, 11 * A, 1 << 20, None) == "E_UNSUPPORTED"
    assert code(attn_plan, dtype=F32, route="tc") == "E_UNSUPPORTED"


def test_python_refusals(lib):
    x = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError):
        layer_norm(x)
    with pytest.raises(ValueError):
        attention(x, x, x)
    with pytest.raises(ValueError):
        rope(x, positions=torch.zeros(3, dtype=torch.int32), inv_freq=torch.ones(4))


def test_frequencies():
    f = rope_frequencies((2, 4), theta=100.0, device="cpu")
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.5, 1.0, 100 ** -0.25, 100 ** -0.5,
                                           100 ** -0.75]))
    f = rope_frequencies((2, 2), theta=100.0, shared=True, device="cpu")
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 100 ** -0.5, 100 ** -0.75]))


def test_the_64_bit_forms_agree_with_autograd():
    R.U[torch.float64], R.TINY[torch.float64] = 2.0 ** -53, 0.0
    x = R.normal(1, (3, 10, 7), torch.float64).requires_grad_()
    w, b = R.normal(2, (10,), torch.float64).requires_grad_(), R.normal(3, (10,), torch.float64).requires_grad_()
    dy = R.normal(4, (3, 10, 7), torch.float64)
    y = torch.nn.functional.layer_norm(x.movedim(1, -1), (10,), w, b, 1e-5).movedim(-1, 1)
    ref = torch.autograd.grad(y, (x, w, b), dy)
    assert torch.allclose(R.layer_norm(x.detach(), w.detach(), b.detach(), 1, 1e-5)[0], y.detach())
    got = R.layer_norm_backward(dy, x.detach(), w.detach(), b.detach(), 1, 1e-5)
    for name, r in zip(("dx", "dweight", "dbias"), ref):
        assert torch.allclose(got[name][0], r), name
    q = R.normal(5, (2, 6, 4, 8), torch.float64).requires_grad_()
    k = R.normal(6, (2, 9, 2, 8), torch.float64).requires_grad_()
    v = R.normal(7, (2, 9, 2, 8), torch.float64).requires_grad_()
    g = R.normal(8, (2, 6, 4, 8), torch.float64)
    kl = torch.tensor([9, 5], dtype=torch.int32)
    ok = R.allowed(2, 6, 9, True, None, kl)
    assert int(ok[1].any(1).sum()) == 5  # the first query of the short sequence sees nothing
    mask = torch.zeros(2, 1, 6, 9, dtype=torch.float64).masked_fill(~ok[:, None], -1e300)
    rep = lambda t: t.transpose(1, 2).repeat_interleave(2, 1)  # noqa: E731
    p = torch.softmax(q.transpose(1, 2) @ rep(k).transpose(2, 3) / 8 ** 0.5 + mask, -1)
    p = p * ok.any(2)[:, None, :, None]
    o = (p @ rep(v)).transpose(1, 2)
    ref = torch.autograd.grad(o, (q, k, v), g)
    got = R.attention(q.detach(), k.detach(), v.detach(), causal=True, kv_lens=kl, dout=g)
    assert torch.allclose(got["out"][0], o.detach())
    for name, r in zip(("dq", "dk", "dv"), ref):
        assert torch.allclose(got[name][0], r), name
