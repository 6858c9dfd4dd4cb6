"""Token-side operators over the C ABI in include/fconv_ops.h: layer norm, rotary positions
with several axes, alone or with the norm of each head, attention, and the gated feed-forward
block, each with its gradient.

As with the convolution, PyTorch only provides device memory and streams: plans are cached by
shape and strides, arguments are checked here and in the library, and every step runs in the
library's CUDA kernels on the current stream of the tensors' device (or the one given), with that
device made current for the call. Outputs carry no gradient function: the backward calls are the
gradients, to be called by hand or from a torch.autograd.Function. Plans are cached by shape: a
program whose keys grow token by token passes one buffer and kv_lens, not a longer view each time.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import Optional, Sequence

from . import FconvError, _lib

I64, I32, F32 = ctypes.c_int64, ctypes.c_int, ctypes.c_float
VP, SZ = ctypes.c_void_p, ctypes.c_size_t
BF16 = 2
PAIRINGS = {"interleaved": 0, "half": 1, "half_per_axis": 2}
ATTN_ROUTES = {"auto": 0, "simple": 1, "tc": 2}
ATTN_ROUTE_NAMES = {v: k for k, v in ATTN_ROUTES.items()}
# Activations of the gated block by the convolution's names; Silu is QuickGelu with alpha 1.
GATES = {None: 0, "Relu": 1, "Sigmoid": 3, "QuickGelu": 8, "Gelu": 10, "FastGelu": 11}


class NormDesc(ctypes.Structure):
    _fields_ = [("dtype", I32), ("param_dtype", I32), ("outer", I64), ("channels", I64),
                ("inner", I64), ("has_weight", I32), ("has_bias", I32), ("eps", F32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("dtype", I32), ("batch", I64), ("len", I64), ("heads_q", I64),
                ("heads_k", I64), ("head_dim", I64), ("q_stride", I64 * 3),
                ("k_stride", I64 * 3), ("q_out_stride", I64 * 3), ("k_out_stride", I64 * 3),
                ("axes", I32), ("section", I64 * 3), ("pairing", I32), ("pos_type", I32),
                ("pos_batch", I64), ("inverse", I32)]


class NormRopeDesc(ctypes.Structure):
    _fields_ = [("dtype", I32), ("param_dtype", I32), ("batch", I64), ("len", I64),
                ("heads_q", I64), ("heads_k", I64), ("head_dim", I64), ("q_stride", I64 * 3),
                ("k_stride", I64 * 3), ("q_out_stride", I64 * 3), ("k_out_stride", I64 * 3),
                ("dq_stride", I64 * 3), ("dk_stride", I64 * 3), ("has_weight", I32),
                ("has_k_weight", I32), ("eps", F32), ("axes", I32), ("section", I64 * 3),
                ("pairing", I32), ("pos_type", I32), ("pos_batch", I64), ("training", I32)]


class MlpDesc(ctypes.Structure):
    _fields_ = [("dtype", I32), ("tokens", I64), ("features", I64), ("hidden", I64),
                ("out_features", I64), ("x_stride", I64), ("y_stride", I64),
                ("gate_stride", I64), ("up_stride", I64), ("down_stride", I64),
                ("dy_stride", I64), ("dx_stride", I64), ("has_b_gate", I32), ("has_b_up", I32),
                ("has_b_down", I32), ("activation", I32), ("alpha", F32), ("training", I32)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("dtype", I32), ("batch", I64), ("len_q", I64), ("len_k", I64),
                ("heads_q", I64), ("heads_kv", I64), ("head_dim", I64), ("q_stride", I64 * 3),
                ("k_stride", I64 * 3), ("v_stride", I64 * 3), ("out_stride", I64 * 3),
                ("dout_stride", I64 * 3), ("dq_stride", I64 * 3), ("dk_stride", I64 * 3),
                ("dv_stride", I64 * 3), ("scale", F32), ("causal", I32), ("has_q_lens", I32),
                ("has_kv_lens", I32), ("training", I32)]


_PROTOS = {
    "fconv_norm_plan_create": [ctypes.POINTER(NormDesc), I32, ctypes.POINTER(VP)],
    "fconv_norm_workspace_size": [VP, ctypes.POINTER(SZ)],
    "fconv_norm_forward": [VP] * 8,
    "fconv_norm_backward": [VP] * 10 + [SZ, VP],
    "fconv_norm_destroy": [VP],
    "fconv_rope_plan_create": [ctypes.POINTER(RopeDesc), I32, ctypes.POINTER(VP)],
    "fconv_rope_run": [VP] * 8,
    "fconv_rope_destroy": [VP],
    "fconv_attn_plan_create": [ctypes.POINTER(AttnDesc), I32, I32, ctypes.POINTER(VP)],
    "fconv_attn_plan_route": [VP, ctypes.POINTER(I32)],
    "fconv_attn_forward_workspace": [VP, ctypes.POINTER(SZ)],
    "fconv_attn_backward_workspace": [VP, ctypes.POINTER(SZ)],
    "fconv_attn_forward": [VP] * 9 + [SZ, VP],
    "fconv_attn_backward": [VP] * 13 + [SZ, VP],
    "fconv_attn_destroy": [VP],
    "fconv_norm_rope_plan_create": [ctypes.POINTER(NormRopeDesc), I32, ctypes.POINTER(VP)],
    "fconv_norm_rope_workspace_size": [VP, ctypes.POINTER(SZ)],
    "fconv_norm_rope_forward": [VP] * 10,
    "fconv_norm_rope_backward": [VP] * 14 + [SZ, VP],
    "fconv_norm_rope_destroy": [VP],
    "fconv_mlp_plan_create": [ctypes.POINTER(MlpDesc), I32, I32, ctypes.POINTER(VP)],
    "fconv_mlp_plan_route": [VP, ctypes.POINTER(I32)],
    "fconv_mlp_forward_workspace": [VP, ctypes.POINTER(SZ)],
    "fconv_mlp_backward_workspace": [VP, ctypes.POINTER(SZ)],
    "fconv_mlp_saved_size": [VP, ctypes.POINTER(SZ)],
    "fconv_mlp_forward": [VP] * 11 + [SZ, VP],
    "fconv_mlp_backward": [VP] * 17 + [SZ, VP],
    "fconv_mlp_destroy": [VP],
    "fconv_ops_check_device": [VP],
    "fconv_ops_status_string": [I32],
}
_ready = None
torch = None  # imported with the first call: the plans alone need no PyTorch


def load() -> ctypes.CDLL:
    """The library with these operators' prototypes set."""
    global _ready
    if _ready is None:
        lib = _lib.load()
        for name, args in _PROTOS.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = I32
            if name.endswith("_destroy"):
                f.restype = None
        lib.fconv_ops_status_string.restype = ctypes.c_char_p
        _ready = lib
    return _ready


def _error(status: int, where: str) -> FconvError:
    return FconvError(status, where, load().fconv_ops_status_string)


def _check(status: int, where: str):
    if status:
        raise _error(status, where)


def _start():
    """First call of an operator: PyTorch and the library."""
    global torch
    import torch as t
    load()
    torch = t


def check_device(stream=None) -> None:
    """Synchronise `stream` (the current device's default one) and raise if a kernel of these
    operators gave up a wait on its device."""
    if torch is None:
        _start()
    check = load().fconv_ops_check_device
    if stream is None:
        status = check(None)
    else:
        status = _run(stream.device.index, check, stream.cuda_stream)
    _check(status, "check_device")


def _code(dtype) -> int:
    code = {torch.float32: _lib.F32, torch.float16: _lib.F16, torch.bfloat16: BF16}.get(dtype)
    if code is None:
        raise _error(14, f"dtype {dtype}")
    return code


class _Plan:
    """Owns a plan of the C library; `kind` names its entry points."""

    kind = ""

    def _create(self, desc, device, *extra):
        self._lib = load()
        self._ptr = VP()
        create = getattr(self._lib, f"fconv_{self.kind}_plan_create")
        _check(create(ctypes.byref(desc), device, *extra, ctypes.byref(self._ptr)),
               f"fconv_{self.kind}_plan_create")

    def _bytes(self, name) -> int:
        n = SZ()
        _check(getattr(self._lib, name)(self._ptr, ctypes.byref(n)), name)
        return n.value

    def __del__(self):
        try:
            if self._ptr:
                getattr(self._lib, f"fconv_{self.kind}_destroy")(self._ptr)
                self._ptr = VP()
        except Exception:
            pass


_KEPT = 1024  # plans a cache holds; a step over ragged batches or a growing cache makes new ones
_keeping = threading.Lock()


def _keep(cache: dict, key, plan):
    """Puts a plan into a cache, whose oldest ones make room."""
    with _keeping:
        while len(cache) >= _KEPT:
            del cache[next(iter(cache))]
        cache[key] = plan
    return plan


def _on_cuda(who: str, device: int, *tensors) -> None:
    """All tensors that are there lie on one CUDA device."""
    if device >= 0:
        for t in tensors:
            if t is not None and t.get_device() != device:
                break
        else:
            return
    raise ValueError(f"{who} runs on tensors of one CUDA device only")


def _on_stream(stream, *tensors):
    """The context of a call on `stream`. The tensors it is given stay allocated until the work
    enqueued there is done, whichever stream they come from."""
    for t in tensors:
        if t is not None and t.get_device() >= 0:  # the call refuses others
            if t.get_device() != stream.device.index:
                raise ValueError("the stream and the tensors must be of one device")
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _current_stream(device: int) -> int:
    """The handle of the device's current stream; the plain handle spares building a Stream
    object (2 us of the call's 10)."""
    return torch._C._cuda_getCurrentRawStream(device)


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _run(device: int, call, *args):
    """call(*args) with the tensors' device current: the library launches on the current one, and
    the handle of a default stream means that device's."""
    if device == _current_device():
        return call(*args)
    with torch.cuda.device(device):
        return call(*args)


def _workspace(nbytes: int, like):
    return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes else None


def _new(like):
    """An uninitialised contiguous tensor of this shape and type (empty_like is the quicker call,
    but keeps the strides of what is not contiguous)."""
    if like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty_like(like, memory_format=torch.contiguous_format)


def _ptr(t):
    return None if t is None else t.data_ptr()


# -------------------------------------------------------------------------------- layer norm

class LayerNormPlan(_Plan):
    """A validated layer norm: x (outer, channels, inner) normalised over channels."""

    kind = "norm"

    def __init__(self, dtype: int, outer: int, channels: int, inner: int = 1, *,
                 param_dtype: Optional[int] = None, has_weight: bool = True,
                 has_bias: bool = True, eps: float = 1e-5, device: int = -1):
        desc = NormDesc(dtype, dtype if param_dtype is None else param_dtype, outer, channels,
                        inner, int(has_weight), int(has_bias), eps)
        self._create(desc, device)
        self.workspace_bytes = self._bytes("fconv_norm_workspace_size")

    def forward_ptrs(self, x, w, b, y, mean, rstd, stream) -> None:
        """Enqueue on raw device pointers (ints or None)."""
        _check(self._lib.fconv_norm_forward(self._ptr, x, w, b, y, mean, rstd, stream),
               "fconv_norm_forward")

    def backward_ptrs(self, dy, x, w, mean, rstd, dx, dw, db, ws, ws_bytes, stream) -> None:
        _check(self._lib.fconv_norm_backward(self._ptr, dy, x, w, mean, rstd, dx, dw, db, ws,
                                             ws_bytes, stream), "fconv_norm_backward")


_norm_plans: dict = {}


def _norm_plan(who, x, weight, bias, axis, eps, device):
    key = (x.dtype, x.shape, axis, None if weight is None else weight.dtype,
           None if bias is None else bias.dtype, eps, device)
    p = _norm_plans.get(key)
    if p is None:
        if not -x.dim() <= axis < x.dim():
            raise ValueError(f"{who}: axis {axis} of a tensor with {x.dim()} axes")
        axis %= x.dim()
        param = weight if weight is not None else bias
        if weight is not None and bias is not None and weight.dtype != bias.dtype:
            raise ValueError(f"{who}: weight and bias must have one type")
        outer, inner = math.prod(x.shape[:axis]), math.prod(x.shape[axis + 1:])
        if inner == 0:  # no positions: as with no rows, nothing to normalise
            outer, inner = 0, 1
        p = LayerNormPlan(_code(x.dtype), outer, x.shape[axis], inner,
                          param_dtype=None if param is None else _code(param.dtype),
                          has_weight=weight is not None, has_bias=bias is not None, eps=eps,
                          device=device)
        p.param_shape = x.shape[axis:axis + 1]
        p.stat_shape = x.shape[:axis] + x.shape[axis + 1:]
        _keep(_norm_plans, key, p)
    for t in (weight, bias):
        if t is not None and (t.shape != p.param_shape or not t.is_contiguous()):
            raise ValueError(f"{who}: weight and bias are vectors of {p.param_shape[0]} values")
    return p


def layer_norm(x, weight=None, bias=None, *, axis: int = -1, eps: float = 1e-5, out=None,
               return_stats: bool = False, stream=None):
    """(x - mean) * rstd * weight + bias over one axis of a contiguous tensor: axis -1 for token
    rows, axis 1 for channels-first features (N, C, D1..Dn). weight and bias have x's type or
    float32. With return_stats also mean and rstd (float32), which the gradient takes. `out`
    may be x."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, x, weight, bias, out):
            return layer_norm(x, weight, bias, axis=axis, eps=eps, out=out,
                              return_stats=return_stats)
    device = x.get_device()
    _on_cuda("layer_norm", device, weight, bias, out)
    p = _norm_plan("layer_norm", x, weight, bias, axis, eps, device)
    if not x.is_contiguous():
        raise ValueError("layer_norm tensors must be contiguous")
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("layer_norm: out must be like x and contiguous")
    mean = rstd = None
    if return_stats:
        mean = torch.empty(p.stat_shape, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _run(device, p.forward_ptrs, x.data_ptr(), _ptr(weight), _ptr(bias), out.data_ptr(),
         _ptr(mean), _ptr(rstd), _current_stream(device))
    return (out, mean, rstd) if return_stats else out


def layer_norm_backward(dy, x, mean, rstd, weight=None, bias=None, *, axis: int = -1,
                        param_grads: bool = True, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm. mean and rstd are the forward pass's; of
    bias only its presence and type matter. dweight and dbias are None for an absent weight or
    bias, or without param_grads."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, dy, x, mean, rstd, weight, bias):
            return layer_norm_backward(dy, x, mean, rstd, weight, bias, axis=axis,
                                       param_grads=param_grads)
    device = x.get_device()
    _on_cuda("layer_norm_backward", device, dy, mean, rstd, weight, bias)
    p = _norm_plan("layer_norm_backward", x, weight, bias, axis, 1e-5, device)
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("layer_norm_backward: dy must be like x")
    for t in (mean, rstd):
        if t.shape != p.stat_shape or t.dtype != torch.float32:
            raise ValueError("layer_norm_backward: mean and rstd are float32 of shape "
                             f"{tuple(p.stat_shape)}")
    if not (dy.is_contiguous() and x.is_contiguous() and mean.is_contiguous()
            and rstd.is_contiguous()):
        raise ValueError("layer_norm_backward tensors must be contiguous")
    dx = torch.empty_like(x)
    dw = torch.empty_like(weight) if weight is not None and param_grads else None
    db = torch.empty_like(bias) if bias is not None and param_grads else None
    n = p.workspace_bytes if dw is not None or db is not None else 0
    ws = _workspace(n, x)
    _run(device, p.backward_ptrs, dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(),
         rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(ws), n, _current_stream(device))
    return dx, dw, db


# ---------------------------------------------------------------------------------- positions


def _heads(who: str, name: str, t) -> None:
    if t.dim() != 4:
        raise ValueError(f"{who}: {name} must be (batch, tokens, heads, head_dim)")
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"{who}: the last axis of {name} must be contiguous")


class RopePlan(_Plan):
    """A validated rotary-position call; strides are (batch, token, head) in elements."""

    kind = "rope"

    def __init__(self, dtype: int, batch: int, length: int, heads_q: int, heads_k: int,
                 head_dim: int, *, q_stride, k_stride=(0, 0, 0), q_out_stride,
                 k_out_stride=(0, 0, 0), sections: Sequence[int], pairing: str = "half",
                 pos_type: int = 0, pos_batch: int = 1, inverse: bool = False,
                 device: int = -1):
        if pairing not in PAIRINGS:
            raise ValueError(f"pairing must be one of {list(PAIRINGS)}")
        sec = list(sections)
        v = (I64 * 3)(*(sec + [0, 0, 0])[:3])
        s3 = lambda s: (I64 * 3)(*s)  # noqa: E731
        desc = RopeDesc(dtype, batch, length, heads_q, heads_k, head_dim, s3(q_stride),
                        s3(k_stride), s3(q_out_stride), s3(k_out_stride), len(sec), v,
                        PAIRINGS[pairing], pos_type, pos_batch, int(inverse))
        self._create(desc, device)

    def run_ptrs(self, q, k, positions, inv_freq, q_out, k_out, stream) -> None:
        _check(self._lib.fconv_rope_run(self._ptr, q, k, positions, inv_freq, q_out, k_out,
                                        stream), "fconv_rope_run")


_rope_plans: dict = {}


def rope_frequencies(sections: Sequence[int], theta: float = 10000.0, shared: bool = False,
                     device="cuda"):
    """inv_freq for `rope`: each axis counts its own frequencies theta^(-i / n) over its n
    pairs, or with `shared` the axes split one sequence over all pairs."""
    if torch is None:
        _start()
    total = sum(sections)
    values = []
    for n in sections:
        base, size = (len(values), total) if shared else (0, n)
        values += [theta ** -((base + i) / size) for i in range(n)]
    return torch.tensor(values, dtype=torch.float32, device=device)


def rope(q, k=None, *, positions, inv_freq, sections: Optional[Sequence[int]] = None,
         pairing: str = "half", inverse: bool = False, out=None, k_out=None, stream=None):
    """Turn the pairs of q (batch, tokens, heads, head_dim), and of k in the same launch, by
    positions * inv_freq. positions is (tokens, axes), (1, tokens, axes) or (batch, tokens,
    axes) of int32, int64 or float32, the last one left out at will for one axis; sections gives
    the pairs of each axis in order (default: all pairs on one axis). `inverse` turns back, which
    is the gradient. q and k may be strided views with a contiguous last axis; out and k_out
    may be q and k. Returns q', or (q', k')."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, q, k, positions, inv_freq, out, k_out):
            return rope(q, k, positions=positions, inv_freq=inv_freq, sections=sections,
                        pairing=pairing, inverse=inverse, out=out, k_out=k_out)
    device = q.get_device()
    _on_cuda("rope", device, k, positions, inv_freq, out, k_out)
    given = out is not None or k_out is not None
    if out is None:
        out = _new(q)
    if k is not None and k_out is None:
        k_out = _new(k)
    sections = None if sections is None else tuple(sections)
    # everything the checks look at is in the key: a call like an earlier one has passed them
    # (new outputs follow from the inputs)
    key = (q.dtype, q.shape, q.stride(), positions.dtype, positions.shape,
           positions.is_contiguous(), inv_freq.dtype, inv_freq.shape, inv_freq.is_contiguous(),
           sections, pairing, inverse, device,
           None if k is None else (k.dtype, k.shape, k.stride()))
    if given:
        key += (out.dtype, out.shape, out.stride(),
                None if k_out is None else (k_out.dtype, k_out.shape, k_out.stride()))
    p = _rope_plans.get(key)
    if p is None:
        p = _keep(_rope_plans, key, _rope_plan(q, k, positions, inv_freq, sections, pairing,
                                               inverse, out, k_out, device))
    _run(device, p.run_ptrs, q.data_ptr(), _ptr(k), positions.data_ptr(), inv_freq.data_ptr(),
         out.data_ptr(), _ptr(k_out), _current_stream(device))
    return out if k is None else (out, k_out)


def _positions(who, q, positions, inv_freq, sections):
    """(sections, code of the positions' type, batches of positions) once they fit q."""
    pos_type = {torch.int32: 0, torch.int64: 1, torch.float32: 2}.get(positions.dtype)
    if pos_type is None:
        raise _error(14, f"positions of {positions.dtype}")
    if sections is None:
        sections = (inv_freq.numel(),)
    shape = tuple(positions.shape)
    if len(sections) == 1 and shape in ((q.shape[1],), (1, q.shape[1]), tuple(q.shape[:2])):
        shape += (1,)
    if len(shape) == 2:
        shape = (1,) + shape
    if (len(shape) != 3 or shape[0] not in (1, q.shape[0]) or shape[1] != q.shape[1]
            or shape[2] != len(sections) or not positions.is_contiguous()):
        raise ValueError(f"{who}: positions must be contiguous (1 or batch, tokens, axes)")
    if (inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous()
            or inv_freq.numel() != sum(sections)):
        raise ValueError(f"{who}: inv_freq must be float32 with one value per pair")
    return sections, pos_type, shape[0]


def _k_like_q(who, q, k):
    _heads(who, "k", k)
    if k.dtype != q.dtype or k.shape[:2] != q.shape[:2] or k.shape[3] != q.shape[3]:
        raise ValueError(f"{who}: k must have q's type, batch, tokens and head_dim")


def _like(who, name, t, like):
    if like is None or t.shape != like.shape or t.dtype != like.dtype:
        raise ValueError(f"{who}: {name} must be like its input")
    _heads(who, name, t)


def _rope_plan(q, k, positions, inv_freq, sections, pairing, inverse, out, k_out, device):
    _heads("rope", "q", q)
    sections, pos_type, pos_batch = _positions("rope", q, positions, inv_freq, sections)
    if k is not None:
        _k_like_q("rope", q, k)
    for name, t, like in (("out", out, q), ("k_out", k_out, k)):
        if t is not None:
            _like("rope", name, t, like)
    b, t, h, d = q.shape
    none = (0, 0, 0)
    return RopePlan(_code(q.dtype), b, t, h, 0 if k is None else k.shape[2], d,
                    q_stride=q.stride()[:3], q_out_stride=out.stride()[:3],
                    k_stride=none if k is None else k.stride()[:3],
                    k_out_stride=none if k is None else k_out.stride()[:3], sections=sections,
                    pairing=pairing, pos_type=pos_type, pos_batch=pos_batch, inverse=inverse,
                    device=device)


# ------------------------------------------------------------------ head norms with positions

class NormRopePlan(_Plan):
    """A validated norm of every head with rotary positions; strides are (batch, token, head) in
    elements. With `training` it is of the backward pass: q_out_stride and k_out_stride are those
    of the incoming gradients, dq_stride and dk_stride of the results."""

    kind = "norm_rope"

    def __init__(self, dtype: int, batch: int, length: int, heads_q: int, heads_k: int,
                 head_dim: int, *, q_stride, q_out_stride, k_stride=(0, 0, 0),
                 k_out_stride=(0, 0, 0), dq_stride=(0, 0, 0), dk_stride=(0, 0, 0),
                 param_dtype: Optional[int] = None, has_weight: bool = True,
                 has_k_weight: bool = False, eps: float = 1e-6, sections: Sequence[int] = (),
                 pairing: str = "half", pos_type: int = 0, pos_batch: int = 1,
                 training: bool = False, device: int = -1):
        if pairing not in PAIRINGS:
            raise ValueError(f"pairing must be one of {list(PAIRINGS)}")
        sec = list(sections)
        s3 = lambda s: (I64 * 3)(*s)  # noqa: E731
        desc = NormRopeDesc(dtype, dtype if param_dtype is None else param_dtype, batch, length,
                            heads_q, heads_k, head_dim, s3(q_stride), s3(k_stride),
                            s3(q_out_stride), s3(k_out_stride), s3(dq_stride), s3(dk_stride),
                            int(has_weight), int(has_k_weight), eps, len(sec),
                            s3((sec + [0, 0, 0])[:3]), PAIRINGS[pairing], pos_type, pos_batch,
                            int(training))
        self._create(desc, device)
        self.workspace_bytes = self._bytes("fconv_norm_rope_workspace_size")

    def forward_ptrs(self, q, k, w, kw, positions, inv_freq, q_out, k_out, stream) -> None:
        _check(self._lib.fconv_norm_rope_forward(self._ptr, q, k, w, kw, positions, inv_freq,
                                                 q_out, k_out, stream), "fconv_norm_rope_forward")

    def backward_ptrs(self, dq_out, dk_out, q, k, w, kw, positions, inv_freq, dq, dk, dw, dkw, ws,
                      ws_bytes, stream) -> None:
        _check(self._lib.fconv_norm_rope_backward(self._ptr, dq_out, dk_out, q, k, w, kw,
                                                  positions, inv_freq, dq, dk, dw, dkw, ws,
                                                  ws_bytes, stream), "fconv_norm_rope_backward")


_norm_rope_plans: dict = {}


def _form(t):
    return None if t is None else (t.dtype, t.shape, t.stride())


def _norm_rope_plan(who, q, k, weight, k_weight, positions, inv_freq, sections, pairing, eps,
                    device, outs, grads=None, given=True):
    """The cached plan of a call. outs: y of q and k, or in the backward pass their gradients;
    grads: the results of the backward pass. Everything the checks look at is in the key, but the
    results where the call made them itself (not `given`): they follow from the inputs."""
    sections = None if sections is None else tuple(sections)
    key = (q.dtype, q.shape, q.stride(), sections, pairing, eps, device)
    if k is not None:
        key += (k.dtype, k.shape, k.stride())
    for t in (weight, k_weight):
        key += (None,) if t is None else (t.dtype, t.shape, t.is_contiguous())
    if positions is not None and inv_freq is not None:
        key += (positions.dtype, positions.shape, positions.is_contiguous(), inv_freq.dtype,
                inv_freq.shape, inv_freq.is_contiguous())
    else:
        key += (positions is None, inv_freq is None)
    if grads is not None:
        key += ("grads", _form(outs[0]), _form(outs[1]))
        if given:
            key += (_form(grads[0]), _form(grads[1]))
    elif given:
        key += (_form(outs[0]), _form(outs[1]))
    p = _norm_rope_plans.get(key)
    if p is not None:
        return p
    _heads(who, "q", q)
    if k is not None:
        _k_like_q(who, q, k)
    if k is None and k_weight is not None:
        raise ValueError(f"{who}: k_weight without k")
    params = {w.dtype for w in (weight, k_weight) if w is not None}
    if len(params) > 1:
        raise ValueError(f"{who}: weight and k_weight must have one type")
    for w in (weight, k_weight):
        if w is not None and (w.shape != q.shape[3:] or not w.is_contiguous()):
            raise ValueError(f"{who}: weights are vectors of {q.shape[3]} values")
    pos_type, pos_batch = 0, 1
    if positions is None:
        if inv_freq is not None or sections:
            raise ValueError(f"{who}: inv_freq and sections go with positions")
        sections = ()
    elif inv_freq is None:
        raise ValueError(f"{who}: positions go with inv_freq")
    else:
        sections, pos_type, pos_batch = _positions(who, q, positions, inv_freq, sections)
    pairs = [outs] if grads is None else [outs, grads]
    for group in pairs:
        for name, t, like in (("q", group[0], q), ("k", group[1], k)):
            if (t is None) != (like is None):
                raise ValueError(f"{who}: k and its gradient go together")
            if t is not None:
                _like(who, f"the output or gradient of {name}", t, like)
    b, n, h, d = q.shape
    st = lambda t: (0, 0, 0) if t is None else t.stride()[:3]  # noqa: E731
    p = NormRopePlan(_code(q.dtype), b, n, h, 0 if k is None else k.shape[2], d,
                     q_stride=st(q), k_stride=st(k), q_out_stride=st(outs[0]),
                     k_out_stride=st(outs[1]),
                     dq_stride=st(None if grads is None else grads[0]),
                     dk_stride=st(None if grads is None else grads[1]),
                     param_dtype=_code(params.pop()) if params else None,
                     has_weight=weight is not None, has_k_weight=k_weight is not None, eps=eps,
                     sections=sections, pairing=pairing, pos_type=pos_type, pos_batch=pos_batch,
                     training=grads is not None, device=device)
    return _keep(_norm_rope_plans, key, p)


def norm_rope(q, k=None, *, weight=None, k_weight=None, positions=None, inv_freq=None,
              sections: Optional[Sequence[int]] = None, pairing: str = "half", eps: float = 1e-6,
              out=None, k_out=None, stream=None):
    """Divide every head of q (batch, tokens, heads, head_dim), and of k in the same launch, by its
    root mean square (sqrt(mean(x^2) + eps)), multiply it by a weight of head_dim values (of q's
    type or float32, one for all heads of q, another for all of k) and turn its pairs by position
    as `rope` does, whose positions, inv_freq, sections and pairing these are. Without positions
    only the norm. head_dim is at most 512. q and k may be strided views with a contiguous last
    axis; out and k_out may be q and k. Returns q', or (q', k')."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, q, k, weight, k_weight, positions, inv_freq, out, k_out):
            return norm_rope(q, k, weight=weight, k_weight=k_weight, positions=positions,
                             inv_freq=inv_freq, sections=sections, pairing=pairing, eps=eps,
                             out=out, k_out=k_out)
    device = q.get_device()
    _on_cuda("norm_rope", device, k, weight, k_weight, positions, inv_freq, out, k_out)
    given = out is not None or k_out is not None
    if out is None:
        out = _new(q)
    if k is not None and k_out is None:
        k_out = _new(k)
    p = _norm_rope_plan("norm_rope", q, k, weight, k_weight, positions, inv_freq, sections,
                        pairing, eps, device, (out, k_out), given=given)
    _run(device, p.forward_ptrs, q.data_ptr(), _ptr(k), _ptr(weight), _ptr(k_weight),
         _ptr(positions), _ptr(inv_freq), out.data_ptr(), _ptr(k_out), _current_stream(device))
    return out if k is None else (out, k_out)


def norm_rope_backward(dout, q, dk_out=None, k=None, *, weight=None, k_weight=None, positions=None,
                       inv_freq=None, sections: Optional[Sequence[int]] = None,
                       pairing: str = "half", eps: float = 1e-6, dq=None, dk=None,
                       param_grads: bool = True, stream=None):
    """Gradients (dq, dk, dweight, dk_weight) of norm_rope from those of its outputs. q and k are
    its inputs, which must still hold what they held then (so not after a call in place); dq and
    dk may be given (dout and dk_out among others, or strided views of one buffer). dk is None
    without k, a weight's gradient without the weight or without param_grads."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, dout, q, dk_out, k, weight, k_weight, positions, inv_freq, dq, dk):
            return norm_rope_backward(dout, q, dk_out, k, weight=weight, k_weight=k_weight,
                                      positions=positions, inv_freq=inv_freq, sections=sections,
                                      pairing=pairing, eps=eps, dq=dq, dk=dk,
                                      param_grads=param_grads)
    device = q.get_device()
    _on_cuda("norm_rope_backward", device, dout, dk_out, k, weight, k_weight, positions, inv_freq,
             dq, dk)
    given = dq is not None or dk is not None
    dq = _new(q) if dq is None else dq
    if k is not None and dk is None:
        dk = _new(k)
    p = _norm_rope_plan("norm_rope_backward", q, k, weight, k_weight, positions, inv_freq,
                        sections, pairing, eps, device, (dout, dk_out), (dq, dk), given)
    dw = torch.empty_like(weight) if weight is not None and param_grads else None
    dkw = torch.empty_like(k_weight) if k_weight is not None and param_grads else None
    n = p.workspace_bytes if dw is not None or dkw is not None else 0
    ws = _workspace(n, q)
    _run(device, p.backward_ptrs, dout.data_ptr(), _ptr(dk_out), q.data_ptr(), _ptr(k),
         _ptr(weight), _ptr(k_weight), _ptr(positions), _ptr(inv_freq), dq.data_ptr(), _ptr(dk),
         _ptr(dw), _ptr(dkw), _ptr(ws), n, _current_stream(device))
    return dq, dk, dw, dkw


# -------------------------------------------------------------------- gated feed-forward block

class MlpPlan(_Plan):
    """A validated gated feed-forward block; strides are those between rows, in elements. A plan
    made with `training` also runs the backward pass."""

    kind = "mlp"

    def __init__(self, dtype: int, tokens: int, features: int, hidden: int, out_features: int, *,
                 x_stride: int, y_stride: int, gate_stride: int, up_stride: int, down_stride: int,
                 dy_stride: int = 0, dx_stride: int = 0, has_b_gate: bool = False,
                 has_b_up: bool = False, has_b_down: bool = False, activation: int = 8,
                 alpha: float = 1.0, training: bool = False, route: str = "auto",
                 device: int = -1):
        desc = MlpDesc(dtype, tokens, features, hidden, out_features, x_stride, y_stride,
                       gate_stride, up_stride, down_stride, dy_stride, dx_stride,
                       int(has_b_gate), int(has_b_up), int(has_b_down), activation, alpha,
                       int(training))
        self._create(desc, device, ATTN_ROUTES[route])
        self.forward_workspace = self._bytes("fconv_mlp_forward_workspace")
        self.backward_workspace = self._bytes("fconv_mlp_backward_workspace")
        self.saved_bytes = self._bytes("fconv_mlp_saved_size")
        r = I32()
        _check(self._lib.fconv_mlp_plan_route(self._ptr, ctypes.byref(r)), "route")
        self.route = ATTN_ROUTE_NAMES[r.value]

    def forward_ptrs(self, x, wg, wu, wd, bg, bu, bd, y, saved, ws, ws_bytes, stream) -> None:
        _check(self._lib.fconv_mlp_forward(self._ptr, x, wg, wu, wd, bg, bu, bd, y, saved, ws,
                                           ws_bytes, stream), "fconv_mlp_forward")

    def backward_ptrs(self, dy, x, wg, wu, wd, bg, bu, saved, dx, dwg, dwu, dwd, dbg, dbu, dbd,
                      ws, ws_bytes, stream) -> None:
        _check(self._lib.fconv_mlp_backward(self._ptr, dy, x, wg, wu, wd, bg, bu, saved, dx, dwg,
                                            dwu, dwd, dbg, dbu, dbd, ws, ws_bytes, stream),
               "fconv_mlp_backward")


_mlp_plans: dict = {}


def _row_stride(who, name, t):
    """The stride between the rows of a tensor seen as (rows, last axis)."""
    if t.dim() < 2 or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{who}: {name} must have rows that are contiguous")
    if t.dim() > 2 and not t.is_contiguous():
        try:
            t = t.view(-1, t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{who}: the rows of {name} must be one stride apart") from None
    if t.dim() > 2:
        return t.shape[-1]
    return t.stride(0)


def _gate(who, activation, params):
    """(code, alpha) of an activation by its name."""
    if activation == "Silu":
        if params is not None:
            raise ValueError(f"{who}: Silu takes no parameters")
        return GATES["QuickGelu"], 1.0
    if activation not in GATES:
        raise ValueError(f"{who}: activation must be Silu or one of {list(GATES)}")
    params = params or ()
    if len(params) > (activation == "QuickGelu"):
        raise ValueError(f"{who}: {activation} takes fewer parameters")
    return GATES[activation], float(params[0]) if params else 1.702


def _mlp_plan(who, x, weights, biases, activation, params, route, device, y, dx=None, given=True):
    """The cached plan of a call. With dx it is a backward pass's, whose dy is y. Everything the
    checks look at is in the key, but a result that the call made itself (not `given`)."""
    wg, wu, wd = weights
    params = None if params is None else tuple(params)  # once: an iterator has no second time
    key = (x.dtype, x.shape, x.stride(), wg.dtype, wg.shape, wg.stride(), wu.dtype, wu.shape,
           wu.stride(), wd.dtype, wd.shape, wd.stride(), activation, params, route, device)
    for b in biases:
        key += (None,) if b is None else (b.dtype, b.shape, b.is_contiguous())
    if dx is not None:
        key += ("grads", _form(y), _form(dx) if given else None)
    elif given:
        key += (_form(y),)
    p = _mlp_plans.get(key)
    if p is not None:
        return p
    for name, w in (("w_gate", wg), ("w_up", wu), ("w_down", wd)):
        if w.dim() != 2 or w.dtype != x.dtype:
            raise ValueError(f"{who}: {name} must be a matrix of x's type")
    if x.dim() < 2:
        raise ValueError(f"{who}: x must be (..., tokens, features)")
    hidden, features = wg.shape
    if wu.shape != wg.shape or x.shape[-1] != features or wd.shape[1] != hidden:
        raise ValueError(f"{who}: w_gate and w_up must be (hidden, {x.shape[-1]}) and w_down "
                         "(out_features, hidden)")
    for name, b, n in zip(("b_gate", "b_up", "b_down"), biases, (hidden, hidden, wd.shape[0])):
        if b is not None and (b.shape != (n,) or b.dtype != x.dtype or not b.is_contiguous()):
            raise ValueError(f"{who}: {name} must be a vector of {n} values of x's type")
    if y.shape != x.shape[:-1] + wd.shape[:1] or y.dtype != x.dtype:
        raise ValueError(f"{who}: the output and its gradient are "
                         f"{tuple(x.shape[:-1] + wd.shape[:1])} of x's type")
    if dx is not None and (dx.shape != x.shape or dx.dtype != x.dtype):
        raise ValueError(f"{who}: dx must be like x")
    code, alpha = _gate(who, activation, params)
    if route not in ATTN_ROUTES:
        raise ValueError(f"{who}: route must be one of {list(ATTN_ROUTES)}")
    out_row = _row_stride(who, "y" if dx is None else "dy", y)
    p = MlpPlan(_code(x.dtype), math.prod(x.shape[:-1]), features, hidden, wd.shape[0],
                x_stride=_row_stride(who, "x", x),
                y_stride=out_row if dx is None else wd.shape[0],
                gate_stride=_row_stride(who, "w_gate", wg),
                up_stride=_row_stride(who, "w_up", wu),
                down_stride=_row_stride(who, "w_down", wd),
                dy_stride=0 if dx is None else out_row,
                dx_stride=0 if dx is None else _row_stride(who, "dx", dx),
                has_b_gate=biases[0] is not None, has_b_up=biases[1] is not None,
                has_b_down=biases[2] is not None, activation=code, alpha=alpha,
                training=dx is not None, route=route, device=device)
    return _keep(_mlp_plans, key, p)


def gated_mlp(x, w_gate, w_up, w_down, *, b_gate=None, b_up=None, b_down=None,
              activation: Optional[str] = "Silu", activation_params=None, out=None,
              return_saved: bool = False, route: str = "auto", stream=None):
    """(act(x w_gate^T + b_gate) * (x w_up^T + b_up)) w_down^T + b_down for x (..., features),
    w_gate and w_up (hidden, features) and w_down (out_features, hidden). Rows are contiguous and
    one stride apart, so gate and up may be halves of one packed weight. activation is Silu, Gelu
    (erf), FastGelu (tanh), QuickGelu (activation_params: alpha), Relu, Sigmoid or None. With
    return_saved also what the gradient takes: both projections in float32, 8 bytes a token and
    hidden value, in an order of the library's own. Over 32 tokens in float16 or bfloat16, tensors
    whose rows are whole units of 16 bytes should start on one: a base off it takes a kernel without
    tcgen05, up to 50 times as long."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, x, w_gate, w_up, w_down, b_gate, b_up, b_down, out):
            return gated_mlp(x, w_gate, w_up, w_down, b_gate=b_gate, b_up=b_up, b_down=b_down,
                             activation=activation, activation_params=activation_params, out=out,
                             return_saved=return_saved, route=route)
    device = x.get_device()
    _on_cuda("gated_mlp", device, w_gate, w_up, w_down, b_gate, b_up, b_down, out)
    given = out is not None
    if out is None:
        if w_down.shape[0] == x.shape[-1]:
            out = _new(x)
        else:
            out = torch.empty(x.shape[:-1] + w_down.shape[:1], dtype=x.dtype, device=x.device)
    p = _mlp_plan("gated_mlp", x, (w_gate, w_up, w_down), (b_gate, b_up, b_down), activation,
                  activation_params, route, device, out, given=given)
    saved = None
    if return_saved:
        saved = torch.empty(p.saved_bytes // 4, dtype=torch.float32, device=x.device)
    n = p.forward_workspace
    ws = _workspace(n, x)
    _run(device, p.forward_ptrs, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
         w_down.data_ptr(), _ptr(b_gate), _ptr(b_up), _ptr(b_down), out.data_ptr(), _ptr(saved),
         _ptr(ws), n, _current_stream(device))
    return (out, saved) if return_saved else out


def gated_mlp_backward(dy, x, w_gate, w_up, w_down, saved=None, *, b_gate=None, b_up=None,
                       b_down=None, activation: Optional[str] = "Silu", activation_params=None,
                       dx=None, param_grads: bool = True, route: str = "auto", stream=None):
    """Gradients (dx, dw_gate, dw_up, dw_down, db_gate, db_up, db_down) of gated_mlp. saved is what
    it returned for these inputs; without it the projections are made again, for two more products
    of x. Of b_down only its presence matters. The gradients of absent biases are None, and without
    param_grads all but dx."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, dy, x, w_gate, w_up, w_down, saved, b_gate, b_up, b_down, dx):
            return gated_mlp_backward(dy, x, w_gate, w_up, w_down, saved, b_gate=b_gate,
                                      b_up=b_up, b_down=b_down, activation=activation,
                                      activation_params=activation_params, dx=dx,
                                      param_grads=param_grads, route=route)
    device = x.get_device()
    _on_cuda("gated_mlp_backward", device, dy, w_gate, w_up, w_down, saved, b_gate, b_up, b_down,
             dx)
    given = dx is not None
    dx = _new(x) if dx is None else dx
    weights, biases = (w_gate, w_up, w_down), (b_gate, b_up, b_down)
    p = _mlp_plan("gated_mlp_backward", x, weights, biases, activation, activation_params, route,
                  device, dy, dx, given)
    n = p.backward_workspace
    if saved is not None:
        if (saved.dtype != torch.float32 or saved.dim() != 1 or not saved.is_contiguous()
                or saved.numel() * 4 != p.saved_bytes):
            raise ValueError("gated_mlp_backward: saved must be what gated_mlp returned")
        n -= p.saved_bytes
    dw, db = [None] * 3, [None] * 3
    if param_grads:
        dw = [_new(w) for w in weights]
        db = [None if b is None else _new(b) for b in biases]
    ws = _workspace(n, x)
    _run(device, p.backward_ptrs, dy.data_ptr(), x.data_ptr(), w_gate.data_ptr(),
         w_up.data_ptr(), w_down.data_ptr(), _ptr(b_gate), _ptr(b_up), _ptr(saved), dx.data_ptr(),
         *map(_ptr, dw), *map(_ptr, db), _ptr(ws), n, _current_stream(device))
    return (dx, *dw, *db)


# ---------------------------------------------------------------------------------- attention

class AttentionPlan(_Plan):
    """A validated attention call; strides are (batch, token, head) in elements. A plan made
    with `training` (and the gradients' strides) also runs the backward pass."""

    kind = "attn"

    def __init__(self, dtype: int, batch: int, len_q: int, len_k: int, heads_q: int,
                 heads_kv: int, head_dim: int, *, q_stride, k_stride, v_stride, out_stride,
                 dout_stride=(0, 0, 0), dq_stride=(0, 0, 0), dk_stride=(0, 0, 0),
                 dv_stride=(0, 0, 0), scale: Optional[float] = None, causal: bool = False,
                 has_q_lens: bool = False, has_kv_lens: bool = False, training: bool = False,
                 route: str = "auto", device: int = -1):
        if scale is None:
            scale = 1.0 / math.sqrt(head_dim) if head_dim > 0 else 1.0
        s3 = lambda s: (I64 * 3)(*s)  # noqa: E731
        desc = AttnDesc(dtype, batch, len_q, len_k, heads_q, heads_kv, head_dim, s3(q_stride),
                        s3(k_stride), s3(v_stride), s3(out_stride), s3(dout_stride),
                        s3(dq_stride), s3(dk_stride), s3(dv_stride), scale, int(causal),
                        int(has_q_lens), int(has_kv_lens), int(training))
        self._create(desc, device, ATTN_ROUTES[route])
        self.forward_workspace = self._bytes("fconv_attn_forward_workspace")
        self.backward_workspace = self._bytes("fconv_attn_backward_workspace")
        r = I32()
        _check(self._lib.fconv_attn_plan_route(self._ptr, ctypes.byref(r)), "route")
        self.route = ATTN_ROUTE_NAMES[r.value]

    def forward_ptrs(self, q, k, v, q_lens, kv_lens, out, lse, ws, ws_bytes, stream) -> None:
        _check(self._lib.fconv_attn_forward(self._ptr, q, k, v, q_lens, kv_lens, out, lse, ws,
                                            ws_bytes, stream), "fconv_attn_forward")

    def backward_ptrs(self, dout, q, k, v, out, lse, q_lens, kv_lens, dq, dk, dv, ws, ws_bytes,
                      stream) -> None:
        _check(self._lib.fconv_attn_backward(self._ptr, dout, q, k, v, out, lse, q_lens, kv_lens,
                                             dq, dk, dv, ws, ws_bytes, stream),
               "fconv_attn_backward")


_attn_plans: dict = {}


def _attn_plan(who, q, k, v, out, causal, scale, q_lens, kv_lens, route, device, grads=None):
    """The cached plan of a call. Everything the checks look at is in the key, so a call like
    an earlier one has passed them. grads: (dout, dq, dk, dv) of a backward pass."""
    key = (q.dtype, k.dtype, v.dtype, out.dtype, q.shape, k.shape, v.shape, out.shape, q.stride(),
           k.stride(), v.stride(), out.stride(), causal, scale, route, device)
    if q_lens is not None or kv_lens is not None:
        for t in (q_lens, kv_lens):
            key += (None,) if t is None else (t.dtype, t.shape, t.is_contiguous())
    if grads is not None:
        for t in grads:
            key += (t.dtype, t.shape, t.stride())
    p = _attn_plans.get(key)
    if p is not None:
        return p
    for name, t in (("q", q), ("k", k), ("v", v)):
        _heads(who, name, t)
    if (k.shape != v.shape or k.dtype != q.dtype or v.dtype != q.dtype
            or k.shape[0] != q.shape[0] or k.shape[3] != q.shape[3]):
        raise ValueError(f"{who}: k and v must be (batch, keys, kv_heads, head_dim) of q's type")
    for name, t in (("q_lens", q_lens), ("kv_lens", kv_lens)):
        if t is not None and (t.dtype != torch.int32 or t.shape != q.shape[:1]
                              or not t.is_contiguous()):
            raise ValueError(f"{who}: {name} must be contiguous int32 with one value a sequence")
    named = [("out", out, q)]
    if grads is not None:
        named += zip(("dout", "dq", "dk", "dv"), grads, (q, q, k, v))
    for name, t, like in named:
        if t.shape != like.shape or t.dtype != like.dtype:
            raise ValueError(f"{who}: {name} has another shape or type than its tensor")
        _heads(who, name, t)
    b, lq, h, d = q.shape
    strides = {}
    if grads is not None:
        strides = {n + "_stride": t.stride()[:3]
                   for n, t in zip(("dout", "dq", "dk", "dv"), grads)}
    p = AttentionPlan(
        _code(q.dtype), b, lq, k.shape[1], h, k.shape[2], d, q_stride=q.stride()[:3],
        k_stride=k.stride()[:3], v_stride=v.stride()[:3], out_stride=out.stride()[:3],
        scale=scale, causal=causal, has_q_lens=q_lens is not None,
        has_kv_lens=kv_lens is not None, training=grads is not None, route=route, device=device,
        **strides)
    p.lse_shape = (b, h, lq)
    return _keep(_attn_plans, key, p)  # whole: another thread may take it from here on


def attention(q, k, v, *, causal: bool = False, scale: Optional[float] = None, q_lens=None,
              kv_lens=None, out=None, return_lse: bool = False, route: str = "auto",
              stream=None):
    """softmax(scale * q k^T) v for q (batch, queries, heads, head_dim) and k, v (batch, keys,
    kv_heads, head_dim); heads is a multiple of kv_heads. scale defaults to head_dim^-1/2.
    q_lens and kv_lens (int32, one value a sequence) cut sequences short; causal lets query i
    see keys up to i + kv_len - q_len. A query that sees no key gives 0. With return_lse also
    the log of the softmax sums (batch, heads, queries) in float32, which the gradient takes."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, q, k, v, q_lens, kv_lens, out):
            return attention(q, k, v, causal=causal, scale=scale, q_lens=q_lens, kv_lens=kv_lens,
                             out=out, return_lse=return_lse, route=route)
    device = q.get_device()
    _on_cuda("attention", device, k, v, q_lens, kv_lens, out)
    if out is None:
        out = _new(q)
    p = _attn_plan("attention", q, k, v, out, causal, scale, q_lens, kv_lens, route, device)
    lse = None
    if return_lse:
        lse = torch.empty(p.lse_shape, dtype=torch.float32, device=q.device)
    n = p.forward_workspace
    ws = _workspace(n, q)
    _run(device, p.forward_ptrs, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(q_lens),
         _ptr(kv_lens), out.data_ptr(), _ptr(lse), _ptr(ws), n, _current_stream(device))
    return (out, lse) if return_lse else out


def attention_backward(dout, q, k, v, out, lse, *, causal: bool = False,
                       scale: Optional[float] = None, q_lens=None, kv_lens=None, dq=None,
                       dk=None, dv=None, route: str = "auto", stream=None):
    """Gradients (dq, dk, dv) of attention, its probabilities made again from lse. out and lse
    are the forward pass's; dq, dk, dv may be given (strided views of one buffer, say)."""
    if torch is None:
        _start()
    if stream is not None:
        with _on_stream(stream, dout, q, k, v, out, lse, q_lens, kv_lens, dq, dk, dv):
            return attention_backward(dout, q, k, v, out, lse, causal=causal, scale=scale,
                                      q_lens=q_lens, kv_lens=kv_lens, dq=dq, dk=dk, dv=dv,
                                      route=route)
    device = q.get_device()
    _on_cuda("attention_backward", device, k, v, dout, out, lse, q_lens, kv_lens, dq, dk, dv)
    dq = _new(q) if dq is None else dq
    dk = _new(k) if dk is None else dk
    dv = _new(v) if dv is None else dv
    p = _attn_plan("attention_backward", q, k, v, out, causal, scale, q_lens, kv_lens, route,
                   device, (dout, dq, dk, dv))
    if lse.shape != p.lse_shape or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("attention_backward: lse must be float32 (batch, heads, queries)")
    n = p.backward_workspace
    ws = _workspace(n, q)
    _run(device, p.backward_ptrs, dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         out.data_ptr(), lse.data_ptr(), _ptr(q_lens), _ptr(kv_lens), dq.data_ptr(),
         dk.data_ptr(), dv.data_ptr(), _ptr(ws), n, _current_stream(device))
    return dq, dk, dv
