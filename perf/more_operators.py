"""The two operators around attention in an encoder block, as measured workloads.

`norm_rope` normalises every head of the queries and keys by its root mean square and turns its
pairs by the token's position, between the fused projection and attention. `gated_mlp` is the
feed-forward block that follows: down(act(gate(x)) * up(x)). A case is one pass through one of
them, forward only ("forward") or forward and backward ("train"). `run` computes a case either in
plain torch operations in 32 bits or through the package's entry points.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases

def _norm_rope(name, direction, dtype, batch, t, h, w, heads_q, heads_k, dim, pairing):
    return {"name": name, "op": "norm_rope", "direction": direction, "dtype": dtype,
            "batch": batch, "t": t, "h": h, "w": w, "heads_q": heads_q, "heads_k": heads_k,
            "dim": dim, "pairing": pairing}


def _mlp(name, direction, dtype, tokens, features, hidden, activation, biases):
    return {"name": name, "op": "gated_mlp", "direction": direction, "dtype": dtype,
            "tokens": tokens, "features": features, "hidden": hidden, "activation": activation,
            "biases": biases}


def listed():
    return [
        # the next token of sixteen sequences being decoded: what a single step waits for
        _norm_rope("heads_token", "forward", "bf16", 16, 1, 1, 1, 32, 8, 128, "half"),
        # queries and keys of one image: two axes, 12 heads of 64
        _norm_rope("heads_image", "forward", "f16", 1, 1, 14, 14, 12, 12, 64, "half"),
        # two clips of 16 frames of 48x48 patches: three axes, shared keys
        _norm_rope("heads_video", "forward", "bf16", 2, 16, 48, 48, 32, 8, 128, "interleaved"),
        # a training batch of images
        _norm_rope("heads_image_train", "train", "f16", 32, 1, 14, 14, 12, 12, 64,
                   "half_per_axis"),
        # training on two clips of 16 frames of 32x32 patches
        _norm_rope("heads_video_train", "train", "bf16", 2, 16, 32, 32, 32, 8, 128, "half"),
        # 32 bits, odd sizes and a head length of 72
        _norm_rope("heads_odd_f32_train", "train", "f32", 3, 1, 9, 37, 16, 16, 72, "interleaved"),
        # one token through a wide block: every weight is read for it
        _mlp("mlp_token", "forward", "bf16", 1, 4096, 10240, "Silu", False),
        # one image through a block of 768 channels, biases on all three projections
        _mlp("mlp_image", "forward", "f16", 196, 768, 2048, "Silu", True),
        # a whole clip at once
        _mlp("mlp_video", "forward", "bf16", 16384, 4096, 10240, "FastGelu", False),
        # a training batch of images with a class token
        _mlp("mlp_image_train", "train", "f16", 32 * 197, 768, 2048, "Silu", True),
        # a training batch of long rows
        _mlp("mlp_rows_train", "train", "bf16", 8192, 4096, 10240, "Silu", False),
        # odd sizes in 32 bits
        _mlp("mlp_odd_f32_train", "train", "f32", 999, 333, 777, "Gelu", True),
    ]


def _span(rng, low, high):
    """An integer between low and high, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    direction = rng.choice(["forward", "train"])
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    if rng.random() < 0.4:
        group, heads_k = rng.choice([1, 1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8, 12])
        dim = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 256])
        t, h, w = rng.choice([1, 1, 2, 5, 16]), _span(rng, 1, 64), _span(rng, 1, 64)
        row = t * h * heads_k * group * dim
        w = max(1, min(w, (1 << 26) // row))
        batch = max(1, min(_span(rng, 1, 32), (1 << 26) // (row * w)))
        return _norm_rope(None, direction, dtype, batch, t, h, w, heads_k * group, heads_k, dim,
                          rng.choice(["half", "interleaved", "half_per_axis"]))
    features, hidden = _span(rng, 24, 4096), _span(rng, 32, 10240)
    if rng.random() < 0.75:
        features, hidden = max(32, features // 32 * 32), max(32, hidden // 32 * 32)
    most = 2e11 if dtype == "f32" else 6e12
    each = (18 if direction == "train" else 6) * features * hidden
    tokens = max(1, min(_span(rng, 1, 16384), int(most / each)))
    return _mlp(None, direction, dtype, tokens, features, hidden,
                rng.choice(["Silu", "Silu", "Gelu", "FastGelu", "Relu", "Sigmoid"]),
                rng.random() < 0.5)


def _sections(case):
    """Pairs of each axis: time, height and width, or height and width of a still image."""
    pairs = case["dim"] // 2
    if case["t"] > 1:
        side = pairs * 3 // 8
        return [pairs - 2 * side, side, side]
    return [pairs // 2, pairs - pairs // 2]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    T = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0):
        x = torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)
        return (x.mul_(scale).add_(shift)).to(T)

    s = {"case": case}
    if case["op"] == "norm_rope":
        b, t, h, w = case["batch"], case["t"], case["h"], case["w"]
        hq, hk, d = case["heads_q"], case["heads_k"], case["dim"]
        tokens = t * h * w
        qkv = normal(b, tokens, hq + 2 * hk, d, scale=1.7)  # what a fused projection gives
        s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
        s["w"], s["kw"] = normal(d, scale=0.2, shift=1.0), normal(d, scale=0.2, shift=1.0)
        grid = [torch.arange(n, device=dev, dtype=torch.int32) for n in (t, h, w)]
        pos = torch.stack(torch.meshgrid(*grid, indexing="ij"), -1).reshape(1, tokens, 3)
        start = torch.randint(0, 1000, (b, 1, 1), generator=g, device=dev, dtype=torch.int32)
        pos = pos.repeat(b, 1, 1)
        pos[:, :, :2] += start  # clips begin at different times, crops at different rows
        s["sections"] = _sections(case)
        s["positions"] = (pos if t > 1 else pos[:, :, 1:]).contiguous()
        s["inv_freq"] = torch.cat([10000.0 ** -(torch.arange(n, device=dev) / n)
                                   for n in s["sections"]]).float()
        if case["direction"] == "train":
            s["dq"], s["dk"] = normal(b, tokens, hq, d), normal(b, tokens, hk, d)
        return s
    n, c, f = case["tokens"], case["features"], case["hidden"]
    s["x"] = normal(n, c)
    both = normal(2 * f, c, scale=c ** -0.5)  # gate and up as one packed projection keeps them
    s["gate"], s["up"] = both[:f], both[f:]
    s["down"] = normal(c, f, scale=f ** -0.5)
    if case["biases"]:
        s["bg"], s["bu"], s["bd"] = (normal(m, scale=0.1) for m in (f, f, c))
    if case["direction"] == "train":
        s["dy"] = normal(n, c)
    return s


# ------------------------------------------------------------------------------ plain forms

def _pairs(case, sections, device):
    """The two element indices of each pair."""
    n = sum(sections)
    p = torch.arange(n, device=device)
    if case["pairing"] == "interleaved":
        return 2 * p, 2 * p + 1
    if case["pairing"] == "half":
        return p, p + n
    size = torch.tensor(sections, device=device)
    first = (size.cumsum(0) - size).repeat_interleave(size)
    low = p + first
    return low, low + size.repeat_interleave(size)


def _plain_norm_rope(s):
    case, sections = s["case"], s["sections"]
    T, dev = s["q"].dtype, s["q"].device
    axis = torch.repeat_interleave(torch.arange(len(sections), device=dev),
                                   torch.tensor(sections, device=dev))
    # angles of far positions need more bits than 32
    angle = s["positions"].double()[:, :, axis] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    low, high = _pairs(case, sections, dev)

    def turn(x, sin):
        a, b = x[..., low], x[..., high]
        y = torch.empty_like(x)
        y[..., low], y[..., high] = a * cos - b * sin, b * cos + a * sin
        return y

    out = {}
    for name, x, w in (("q", s["q"], s["w"]), ("k", s["k"], s["kw"])):
        x, wf = x.float(), w.float()
        r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        n = x * r
        out[name] = turn(n * wf, sin).to(T)
        if case["direction"] == "train":
            g = turn(s["d" + name].float(), -sin)
            a = g * wf
            out["d" + name] = (r * (a - n * (a * n).mean(-1, keepdim=True))).to(T)
            out["dw" + name] = (g * n).sum((0, 1, 2)).to(T)
    return out


_INV_SQRT2 = 0.7071067811865476
_INV_SQRT_2PI = 0.3989422804014327
_TANH_C = 0.7978845608028654


def _act(kind, v):
    """The activation and its derivative."""
    if kind == "Relu":
        on = (v > 0).to(v.dtype)
        return v * on, on
    if kind == "Sigmoid":
        p = 1.0 / (1.0 + (-v).exp())
        return p, p * (1.0 - p)
    if kind == "Silu":
        p = 1.0 / (1.0 + (-v).exp())
        return v * p, p * (1.0 + v * (1.0 - p))
    if kind == "Gelu":
        phi = 0.5 * (1.0 + (v * _INV_SQRT2).erf())
        return v * phi, phi + v * _INV_SQRT_2PI * (-0.5 * v * v).exp()
    t = (_TANH_C * (v + 0.044715 * v * v * v)).tanh()
    slope = _TANH_C * (1.0 + 3 * 0.044715 * v * v)
    return 0.5 * v * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * slope


def _plain_mlp(s):
    case, T = s["case"], s["x"].dtype
    x, wg, wu, wd = (s[n].float() for n in ("x", "gate", "up", "down"))
    g, u = x @ wg.t(), x @ wu.t()
    if case["biases"]:
        g, u = g + s["bg"].float(), u + s["bu"].float()
    a, da = _act(case["activation"], g)
    h = a * u
    y = h @ wd.t()
    if case["biases"]:
        y = y + s["bd"].float()
    out = {"y": y.to(T)}
    if case["direction"] == "train":
        dy = s["dy"].float()
        dh = dy @ wd
        dg, du = dh * u * da, dh * a
        out["dx"] = (dg @ wg + du @ wu).to(T)
        out["dgate"], out["dup"] = (dg.t() @ x).to(T), (du.t() @ x).to(T)
        out["ddown"] = (dy.t() @ h).to(T)
        if case["biases"]:
            out["dbg"], out["dbu"], out["dbd"] = (v.sum(0).to(T) for v in (dg, du, dy))
    return out


# -------------------------------------------------------------------------------------- run

def _own_run(s):
    import activation_implicit_gemm_gb300 as fc
    case = s["case"]
    train = case["direction"] == "train"
    if case["op"] == "norm_rope":
        how = dict(weight=s["w"], k_weight=s["kw"], positions=s["positions"],
                   inv_freq=s["inv_freq"], sections=s["sections"], pairing=case["pairing"],
                   eps=1e-6)
        q, k = fc.norm_rope(s["q"], s["k"], **how)
        out = {"q": q, "k": k}
        if train:
            dq, dk, dw, dkw = fc.norm_rope_backward(s["dq"], s["q"], s["dk"], s["k"], **how)
            out.update(dq=dq, dwq=dw, dk=dk, dwk=dkw)
        return out
    weights = (s["gate"], s["up"], s["down"])
    how = dict(b_gate=s.get("bg"), b_up=s.get("bu"), b_down=s.get("bd"),
               activation=case["activation"])
    if not train:
        return {"y": fc.gated_mlp(s["x"], *weights, **how)}
    y, saved = fc.gated_mlp(s["x"], *weights, **how, return_saved=True)
    dx, dgate, dup, ddown, dbg, dbu, dbd = fc.gated_mlp_backward(s["dy"], s["x"], *weights, saved,
                                                                 **how)
    out = {"y": y, "dx": dx, "dgate": dgate, "dup": dup, "ddown": ddown}
    if case["biases"]:
        out.update(dbg=dbg, dbu=dbu, dbd=dbd)
    return out


def run(state):
    if own:
        return _own_run(state)
    if state["case"]["op"] == "norm_rope":
        return _plain_norm_rope(state)
    return _plain_mlp(state)


# ------------------------------------------------------------------------------------- work

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    train = case["direction"] == "train"
    if case["op"] == "norm_rope":
        tokens = case["batch"] * case["t"] * case["h"] * case["w"]
        n = tokens * (case["heads_q"] + case["heads_k"]) * case["dim"]
        axes = 3 if case["t"] > 1 else 2
        params = 4 * (case["dim"] // 2) + (2 if train else 1) * 2 * case["dim"] * e
        # x in, y out; in training also dy in, dx out
        return {"bytes": (4 if train else 2) * n * e + 4 * tokens * axes + params,
                "flops": (22 if train else 8) * n}
    n, c, f = case["tokens"], case["features"], case["hidden"]
    params = 3 * c * f + (2 * f + c if case["biases"] else 0)
    if train:  # x, dy in, y, dx out; weights in, their gradients out
        return {"bytes": e * (4 * n * c + 2 * params), "flops": 18 * n * c * f}
    return {"bytes": e * (2 * n * c + params), "flops": 6 * n * c * f}


# ------------------------------------------------------------------------------------ exact

def _exact_norm_rope(s):
    case, sections = s["case"], s["sections"]
    D = case["dim"]
    pos, freq = s["positions"].double(), s["inv_freq"].double()
    n = sum(sections)
    ends = [sum(sections[:a + 1]) for a in range(len(sections))]
    axis = [next(a for a, e in enumerate(ends) if p < e) for p in range(n)]

    def members(p):
        start = ends[axis[p]] - sections[axis[p]]
        return {"half": (p, p + n), "interleaved": (2 * p, 2 * p + 1),
                "half_per_axis": (start + p, start + p + sections[axis[p]])}[case["pairing"]]

    def spin(x, sign):
        y = x.clone()
        for p in range(n):
            lo, hi = members(p)
            at = sign * pos[..., axis[p]] * freq[p]
            z = torch.complex(x[..., lo], x[..., hi])
            z = z * torch.polar(torch.ones_like(at), at)[..., None]
            y[..., lo], y[..., hi] = z.real, z.imag
        return y

    out = {}
    for name, key in (("q", "w"), ("k", "kw")):
        x, w = s[name].double(), s[key].double()
        rms = torch.sqrt(torch.linalg.vecdot(x, x) / D + 1e-6).unsqueeze(-1)
        z = x / rms
        out[name] = spin(z * w, 1.0)
        if case["direction"] == "train":
            back = spin(s["d" + name].double(), -1.0)
            out["dw" + name] = torch.einsum("blhd,blhd->d", back, z)
            dz = back * w
            out["d" + name] = (dz - z * (torch.linalg.vecdot(dz, z) / D).unsqueeze(-1)) / rms
    return out


def _exact_mlp(s):
    case = s["case"]
    f64 = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    x, G, U, D = f64["x"], f64["gate"], f64["up"], f64["down"]
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    bg, bu, bd = (f64.get(n, zero) for n in ("bg", "bu", "bd"))
    train = case["direction"] == "train"
    g = torch.einsum("nc,fc->nf", x, G) + bg
    u = torch.einsum("nc,fc->nf", x, U) + bu
    kind = case["activation"]
    if train:
        g.requires_grad_()
    with torch.enable_grad():  # the slope by differentiation, not by its formula
        if kind == "Silu":
            a = g * torch.sigmoid(g)
        elif kind == "Sigmoid":
            a = torch.sigmoid(g)
        elif kind == "Relu":
            a = torch.clamp(g, min=0.0)
        elif kind == "Gelu":
            a = 0.5 * g * torch.erfc(-g / math.sqrt(2.0))
        else:  # (1 + tanh z) / 2 is the sigmoid of 2 z
            a = g * torch.sigmoid(math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3))
        slope = torch.autograd.grad(a.sum(), g)[0] if train else None
    a, g = a.detach(), g.detach()
    h = u * a
    out = {"y": torch.einsum("nf,cf->nc", h, D) + bd}
    if train:
        dy = f64["dy"]
        dh = torch.einsum("nc,cf->nf", dy, D)
        out["ddown"] = torch.einsum("nc,nf->cf", dy, h)
        du = dh * a
        dg = dh.mul_(u).mul_(slope)
        out["dx"] = torch.einsum("nf,fc->nc", dg, G) + torch.einsum("nf,fc->nc", du, U)
        out["dgate"] = torch.einsum("nf,nc->fc", dg, x)
        out["dup"] = torch.einsum("nf,nc->fc", du, x)
        if case["biases"]:
            ones = torch.ones_like(x[:, 0])
            out["dbg"], out["dbu"], out["dbd"] = ones @ dg, ones @ du, ones @ dy
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(s)
    if work(case)["flops"] > 8e12:  # over about 20 seconds in 64 bits
        return None
    return _exact_mlp(s)
