"""The Python side of the token-side operators, without a GPU: what it accepts, what it does
around a call and what it says when it refuses."""
import pytest
import torch

from activation_implicit_gemm_gb300 import _build, _ops


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    _ops._start()


# ------------------------------------------------------------------------ forms of positions

def rope_plan(shape, sections, batch=2, tokens=6):
    q = torch.zeros(batch, tokens, 3, 16)
    freq = torch.ones(8 if sections is None else sum(sections))
    return _ops._rope_plan(q, None, torch.zeros(shape, dtype=torch.int32), freq, sections, "half",
                           False, q, None, -1)


@pytest.mark.parametrize("shape", [(6,), (6, 1), (1, 6), (2, 6), (1, 6, 1), (2, 6, 1)])
@pytest.mark.parametrize("sections", [None, (8,)])
def test_positions_of_one_axis(shape, sections):
    rope_plan(shape, sections)


@pytest.mark.parametrize("shape", [(6, 2), (1, 6, 2), (2, 6, 2)])
def test_positions_of_two_axes(shape):
    rope_plan(shape, (3, 5))


@pytest.mark.parametrize("shape,sections", [
    ((5,), None), ((3, 6), None), ((6, 2), None), ((2, 6, 2), None), ((6,), (3, 5)),
    ((2, 6), (3, 5)), ((1, 6), (3, 5)), ((6, 3), (3, 5)), ((3, 6, 2), (3, 5)), ((), None),
    ((1, 2, 6, 1), None)])
def test_positions_that_do_not_fit(shape, sections):
    with pytest.raises(ValueError, match="positions"):
        rope_plan(shape, sections)


def test_positions_of_one_token_a_sequence():
    """Two axes of length one are the same thing either way round."""
    for shape in ((4,), (4, 1), (1, 4)):
        rope_plan(shape, None, batch=1, tokens=4)
    for shape in ((1,), (1, 1), (4, 1), (1, 1, 1), (4, 1, 1)):
        rope_plan(shape, None, batch=4, tokens=1)


# ------------------------------------------------------------------- the tensors' own device

class OnDevice1(torch.Tensor):
    """A tensor that says it lies on the second GPU."""

    def get_device(self):
        return 1


def on_device_1(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice1)


class Switch:
    """Stands in for torch.cuda.device: notes the device that is current while it is entered."""
    current = 0

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        self.before, Switch.current = Switch.current, self.device

    def __exit__(self, *a):
        Switch.current = self.before


def test_the_tensors_device_is_current_in_a_call(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", Switch)
    monkeypatch.setattr(_ops, "_current_device", lambda: Switch.current)
    seen = []
    for device in (1, 0, 1):
        _ops._run(device, lambda *a: seen.append((Switch.current, a)), 5, 6)
    assert seen == [(1, (5, 6)), (0, (5, 6)), (1, (5, 6))] and Switch.current == 0


def test_every_call_runs_on_its_tensors_device(monkeypatch):
    calls = []
    monkeypatch.setattr(_ops, "_run", lambda device, call, *a: calls.append((device, call.__name__)))
    monkeypatch.setattr(_ops, "_current_stream", lambda device: 0)
    x, w = on_device_1(4, 8), on_device_1(8)
    stat = on_device_1(4)
    _ops.layer_norm(x, w, w)
    _ops.layer_norm_backward(x, x, stat, stat, w, w)
    q = on_device_1(1, 3, 2, 8)
    _ops.rope(q, q, positions=on_device_1(3, dtype=torch.int32), inv_freq=on_device_1(4))
    _ops.attention(q, q, q)
    _ops.attention_backward(q, q, q, q, q, on_device_1(1, 2, 3))
    assert calls == [(1, "forward_ptrs"), (1, "backward_ptrs"), (1, "run_ptrs"),
                     (1, "forward_ptrs"), (1, "backward_ptrs")]


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 0)

    x = on_device_1(4, 8)
    q = on_device_1(1, 3, 2, 8)
    for call in (lambda: _ops.layer_norm(x, stream=Stream()),
                 lambda: _ops.attention(q, q, q, stream=Stream())):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_check_device_looks_at_the_streams_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", Switch)
    monkeypatch.setattr(_ops, "_current_device", lambda: Switch.current)
    seen = []

    class Lib:
        @staticmethod
        def fconv_ops_check_device(stream):
            seen.append((Switch.current, stream))
            return 0

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 77

    monkeypatch.setattr(_ops, "load", lambda: Lib)
    _ops.check_device(Stream())
    _ops.check_device()
    assert seen == [(1, 77), (0, None)]


def test_a_convolution_runs_on_its_tensors_device(monkeypatch):
    from activation_implicit_gemm_gb300 import FusedConvPlan
    monkeypatch.setattr(torch.cuda, "device", Switch)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: Switch.current)

    class Stream:
        cuda_stream = 5

    x, w = on_device_1(1, 3, 8, 8), on_device_1(4, 3, 3, 3)
    plan = FusedConvPlan(0, x.shape, w.shape)
    seen = []
    monkeypatch.setattr(plan, "run_ptrs", lambda *a: seen.append((Switch.current, a[-1])))
    plan.run(x, w, stream=Stream())
    assert seen == [(1, 5)] and Switch.current == 0


# ------------------------------------------------------------------------------ cached plans

class Watched(dict):
    """A plan cache that looks at what is put into it."""

    def __init__(self, ready):
        super().__init__()
        self.ready = ready

    def __setitem__(self, key, plan):
        assert self.ready(plan)
        super().__setitem__(key, plan)


def attn_plan(keys, **kw):
    q, k = torch.zeros(1, 2, 4, 16), torch.zeros(1, keys, 2, 16)
    return _ops._attn_plan("attention", q, k, k, q, False, None, None, None, "auto", -1, **kw)


def norm_plan(rows):
    return _ops._norm_plan("layer_norm", torch.zeros(rows, 8), None, None, -1, 1e-5, -1)


def test_a_plan_is_whole_when_other_threads_can_see_it(monkeypatch):
    monkeypatch.setattr(_ops, "_attn_plans", Watched(lambda p: p.lse_shape == (1, 4, 2)))
    monkeypatch.setattr(_ops, "_norm_plans", Watched(lambda p: p.param_shape and p.stat_shape))
    assert attn_plan(5) is attn_plan(5) and len(_ops._attn_plans) == 1
    assert norm_plan(3) is norm_plan(3) and len(_ops._norm_plans) == 1


def rope_call_plan(tokens):
    """A plan as rope() makes and keeps it."""
    q = on_device_1(1, tokens, 2, 8)
    _ops.rope(q, positions=on_device_1(tokens, dtype=torch.int32), inv_freq=on_device_1(4))


def test_the_caches_drop_their_oldest_plans(monkeypatch):
    monkeypatch.setattr(_ops, "_run", lambda *a: None)
    monkeypatch.setattr(_ops, "_current_stream", lambda device: 0)
    monkeypatch.setattr(_ops, "_KEPT", 4)
    for name in ("_attn_plans", "_norm_plans", "_rope_plans"):
        monkeypatch.setattr(_ops, name, {})
    for n in range(1, 12):  # keys that grow by one, as a decoder's do
        attn_plan(n)
        norm_plan(n)
        rope_call_plan(n)
    for cache in (_ops._attn_plans, _ops._norm_plans, _ops._rope_plans):
        assert len(cache) == 4
    newest = list(_ops._attn_plans.values())
    assert [attn_plan(n) for n in range(8, 12)] == newest  # the newest are kept
    assert attn_plan(1) is attn_plan(1) and len(_ops._attn_plans) == 4


def test_threads_share_the_caches(monkeypatch):
    import threading
    monkeypatch.setattr(_ops, "_KEPT", 3)
    monkeypatch.setattr(_ops, "_attn_plans", {})
    failed = []

    def work(seed):
        try:
            for i in range(200):
                assert attn_plan(1 + (i * seed) % 13).lse_shape == (1, 4, 2)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in (1, 2, 3, 5, 7, 11)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(_ops._attn_plans) <= 3


# -------------------------------------------------------------------------- texts of refusals

def test_a_refusal_says_what_the_operators_call_it():
    from activation_implicit_gemm_gb300 import AttentionPlan, FconvError, FusedConvPlan, LayerNormPlan

    def text(call, *a, **kw):
        with pytest.raises(FconvError) as e:
            call(*a, **kw)
        return e.value.code, str(e.value)

    attribute = "an attribute has a value outside its range"
    assert text(LayerNormPlan, 1, 3, 40, eps=-1.0) == (
        "E_ATTR_VALUE", f"fconv_norm_plan_create: E_ATTR_VALUE ({attribute})")
    s = dict(q_stride=(0, 0, 0), k_stride=(0, 0, 0), v_stride=(0, 0, 0), out_stride=(0, 0, 0))
    assert attribute in text(AttentionPlan, 1, 1, 1, 1, 1, 1, 1, scale=-2.0, **s)[1]
    A = 0x10000  # made-up addresses: never read on these paths
    norm = LayerNormPlan(1, 3, 40)
    assert "an output must not be an input" in text(
        norm.forward_ptrs, A, 2 * A, 3 * A, 2 * A, None, None, None)[1]
    assert "as its type or route needs" in text(
        norm.forward_ptrs, A + 1, 2 * A, 3 * A, 4 * A, None, None, None)[1]
    bare = LayerNormPlan(1, 3, 40, has_weight=False, has_bias=False)
    assert "that the plan does not have" in text(
        bare.forward_ptrs, A, 2 * A, None, 4 * A, None, None, None)[1]
    # a convolution's refusals keep their own
    assert "strides/dilations must be >= 1" in text(
        FusedConvPlan, 1, (1, 3, 8, 8), (4, 3, 3, 3), strides=[0, 1])[1]


# ----------------------------------------------------------------- reports of waits given up

def test_check_device_is_part_of_the_package():
    import activation_implicit_gemm_gb300 as fc
    assert fc.check_device is _ops.check_device and "check_device" in fc.__all__


def test_check_device_raises_what_a_kernel_reported(monkeypatch):
    import activation_implicit_gemm_gb300 as fc
    lib = _ops.load()

    class Lib:
        fconv_ops_status_string = staticmethod(lib.fconv_ops_status_string)

        @staticmethod
        def fconv_ops_check_device(stream):
            return 16

    monkeypatch.setattr(_ops, "load", lambda: Lib)
    with pytest.raises(fc.FconvError, match="E_DEVICE_TIMEOUT.*gave up a bounded wait"):
        fc.check_device()
