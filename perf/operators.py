"""The token-side operators next to the convolutions, as measured workloads.

A vision or video encoder whose patch embedding is a FusedConv goes on with layer norm
(over channels-first stem features or over token rows), rotary positions with one axis per
spatial dimension, and attention, each with its gradient. A case is one pass through one of
them: `layer_norm`, `rope` or `attention`, forward only ("forward") or forward and backward
("train"). `run` computes a case either in plain torch operations in 32 bits or through the
package's entry points.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases

def _norm(name, direction, dtype, outer, channels, inner, params):
    return {"name": name, "op": "layer_norm", "direction": direction, "dtype": dtype,
            "outer": outer, "channels": channels, "inner": inner, "params": params}


def _rope(name, dtype, batch, t, h, w, heads_q, heads_k, dim, pairing):
    return {"name": name, "op": "rope", "direction": "forward", "dtype": dtype, "batch": batch,
            "t": t, "h": h, "w": w, "heads_q": heads_q, "heads_k": heads_k, "dim": dim,
            "pairing": pairing}


def _attn(name, direction, dtype, batch, len_q, len_k, heads_q, heads_kv, dim, causal, ragged):
    return {"name": name, "op": "attention", "direction": direction, "dtype": dtype,
            "batch": batch, "len_q": len_q, "len_k": len_k, "heads_q": heads_q,
            "heads_kv": heads_kv, "dim": dim, "causal": causal, "ragged": ragged}


def listed():
    return [
        # one 224x224 image in 16x16 patches, 768 channels: the latency of a single request
        _norm("norm_image", "forward", "f16", 196, 768, 1, "f16"),
        # a training batch of the 56x56 stem features, channels first, 128 channels
        _norm("norm_stem_train", "train", "f16", 32, 128, 56 * 56, "f16"),
        # a training batch of wide token rows, parameters kept in 32 bits
        _norm("norm_rows_train", "train", "bf16", 32768, 4096, 1, "f32"),
        # an odd row length (no 16-byte rows) in 32 bits
        _norm("norm_odd_f32_train", "train", "f32", 5001, 1001, 1, "f32"),
        # queries and keys of one image: two axes, 12 heads of 64
        _rope("rope_image", "f16", 1, 1, 14, 14, 12, 12, 64, "half"),
        # queries and keys of two clips of 16 frames of 48x48 patches: three axes, shared keys
        _rope("rope_video", "bf16", 2, 16, 48, 48, 32, 8, 128, "interleaved"),
        # one image through one attention layer: 196 tokens
        _attn("attn_image", "forward", "f16", 1, 196, 196, 12, 12, 64, False, False),
        # pooling by one query token a sequence over long, ragged sequences; shared heads
        _attn("attn_pool", "forward", "bf16", 16, 1, 8192, 32, 8, 128, False, True),
        # a whole clip at once
        _attn("attn_video", "forward", "bf16", 1, 16384, 16384, 16, 16, 128, False, False),
        # a training batch of images with a class token: 197 tokens
        _attn("attn_image_train", "train", "f16", 32, 197, 197, 12, 12, 64, False, False),
        # training on packed-to-length sequences in causal order, shared heads, ragged lengths
        _attn("attn_causal_train", "train", "bf16", 2, 4096, 4096, 32, 8, 128, True, True),
        # cross attention in 32 bits with odd sizes and a head length of 72
        _attn("attn_cross_f32_train", "train", "f32", 3, 333, 777, 16, 16, 72, False, True),
    ]


def _span(rng, low, high):
    """An integer between low and high, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["norm_rows", "norm_first", "rope", "attn", "attn", "attn_train",
                       "attn_train"])
    if kind == "norm_rows":
        channels = _span(rng, 32, 8192)
        if rng.random() < 0.6:
            channels = max(32, channels // 32 * 32)
        dtype = rng.choice(["f16", "bf16", "f32"])
        outer = min(_span(rng, 1, 65536), (1 << (25 if dtype == "f32" else 26)) // channels)
        return _norm(None, rng.choice(["forward", "train"]), dtype, outer, channels, 1,
                     rng.choice([dtype, "f32"]))
    if kind == "norm_first":
        channels = _span(rng, 24, 1024)
        inner = _span(rng, 7, 112) * _span(rng, 7, 112)
        outer = min(_span(rng, 1, 64), max(1, (1 << 25) // (channels * inner)))
        dtype = rng.choice(["f16", "bf16", "f32"])
        return _norm(None, rng.choice(["forward", "train"]), dtype, outer, channels, inner,
                     rng.choice([dtype, "f32"]))
    if kind == "rope":
        group, heads_k = rng.choice([1, 1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8, 12])
        dim = rng.choice([32, 64, 72, 80, 96, 128])
        t, h, w = rng.choice([1, 1, 2, 5, 16]), _span(rng, 1, 64), _span(rng, 1, 64)
        row = t * h * heads_k * group * dim
        w = max(1, min(w, (1 << 26) // row))
        batch = max(1, min(_span(rng, 1, 32), (1 << 26) // (row * w)))
        return _rope(None, rng.choice(["f16", "bf16", "f32"]), batch, t, h, w, heads_k * group,
                     heads_k, dim, rng.choice(["half", "interleaved", "half_per_axis"]))
    group, heads_kv = rng.choice([1, 1, 1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    heads = group * heads_kv
    dtype = rng.choice(["f16", "f16", "f16", "bf16", "bf16", "bf16", "bf16", "f32"])
    top = 2048 if dtype == "f32" else 8192
    low = 16 if kind == "attn_train" else 1  # with one key every gradient of the scores is zero
    len_k = _span(rng, low, top)
    len_q = len_k if rng.random() < 0.5 else _span(rng, 1, top) if kind == "attn_train" \
        else rng.choice([1, 1, _span(rng, 1, top)])
    most = (1 << 29) // (4 if dtype == "f32" else 1)
    if heads * len_q * len_k > most:
        shrink = math.sqrt(most / (heads * len_q * len_k))
        same = len_q == len_k
        len_k = int(len_k * shrink)
        len_q = len_k if same else max(1, int(len_q * shrink))
    batch = max(1, min(_span(rng, 1, 32), most // (heads * len_q * len_k)))
    return _attn(None, "forward" if kind == "attn" else "train", dtype, batch, len_q, len_k,
                 heads, heads_kv, rng.choice([32, 64, 64, 72, 80, 96, 128, 128]),
                 rng.random() < 0.4, rng.random() < 0.4)


def _lens(case):
    """The valid tokens of each sequence of a ragged batch: (of queries, of keys). The first
    sequence is full, and in a batch of three or more the last one has no keys at all."""
    b, lq, lk = case["batch"], case["len_q"], case["len_k"]
    if not case["ragged"]:
        return [lq] * b, [lk] * b
    ks = [lk - (i * lk * 5) // (b * 7) - i % 2 * min(3, lk // 8) for i in range(b)]
    if b >= 3:
        ks[-1] = 0
    qs = list(ks) if lq == lk else [lq] * b
    return qs, ks


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

    def normal(*shape, scale=1.0, shift=0.0, dtype=T):
        x = torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)
        return (x.mul_(scale).add_(shift)).to(dtype)

    s = {"case": case}
    if case["op"] == "layer_norm":
        n, c, i = case["outer"], case["channels"], case["inner"]
        shape = (n, c) if i == 1 else (n, c, i)
        P = _TYPES[case["params"]]
        s["x"] = normal(*shape, scale=1.5, shift=0.3)
        s["weight"] = normal(c, scale=0.2, shift=1.0, dtype=P)
        s["bias"] = normal(c, scale=0.1, dtype=P)
        if case["direction"] == "train":
            s["dy"] = normal(*shape)
    elif case["op"] == "rope":
        b, t, h, w = case["batch"], case["t"], case["h"], case["w"]
        hq, hk, d = case["heads_q"], case["heads_k"], case["dim"]
        qkv = normal(b, t * h * w, hq + 2 * hk, d)  # what a fused projection gives
        s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
        grid = [torch.arange(n, device=dev, dtype=torch.int32) for n in (t, h, w)]
        pos = torch.stack(torch.meshgrid(*grid, indexing="ij"), -1).reshape(1, t * h * w, 3)
        start = torch.randint(0, 1000, (b, 1, 1), generator=g, device=dev, dtype=torch.int32)
        pos = pos.repeat(b, 1, 1)
        pos[:, :, :1] += start  # clips begin at different times
        s["sections"] = _sections(case)
        s["positions"] = (pos if case["t"] > 1 else pos[:, :, 1:]).contiguous()
        s["inv_freq"] = torch.cat([10000.0 ** -(torch.arange(n, device=dev) / n)
                                   for n in s["sections"]]).float()
    else:
        b, lq, lk = case["batch"], case["len_q"], case["len_k"]
        hq, hk, d = case["heads_q"], case["heads_kv"], case["dim"]
        if lq == lk:
            qkv = normal(b, lq, hq + 2 * hk, d)
            s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
        else:
            kv = normal(b, lk, 2 * hk, d)
            s["q"], s["k"], s["v"] = normal(b, lq, hq, d), kv[:, :, :hk], kv[:, :, hk:]
        if case["ragged"]:
            qs, ks = _lens(case)
            s["q_lens"] = torch.tensor(qs, device=dev, dtype=torch.int32)
            s["kv_lens"] = torch.tensor(ks, device=dev, dtype=torch.int32)
        if case["direction"] == "train":
            s["dout"] = normal(b, lq, hq, d)
    return s


# ------------------------------------------------------------------------------ plain forms

def _plain_norm(s):
    case = s["case"]
    x, T, P = s["x"], s["x"].dtype, s["weight"].dtype
    tail = (1,) * (x.dim() - 2)
    xf, w, b = x.float(), s["weight"].float().view(-1, *tail), s["bias"].float().view(-1, *tail)
    mean = xf.mean(1, keepdim=True)
    xc = xf - mean
    rstd = (xc.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    xhat = xc * rstd
    out = {"y": (xhat * w + b).to(T)}
    if case["direction"] == "train":
        dy = s["dy"].float()
        dims = [0] + list(range(2, x.dim()))
        gx = dy * w
        dx = rstd * (gx - gx.mean(1, keepdim=True) - xhat * (gx * xhat).mean(1, keepdim=True))
        out["dx"] = dx.to(T)
        out["dweight"] = (dy * xhat).sum(dims).to(P)
        out["dbias"] = dy.sum(dims).to(P)
    return out


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


def _plain_rope(s):
    case, sections = s["case"], s["sections"]
    dev = s["q"].device
    axis = torch.repeat_interleave(torch.arange(len(sections), device=dev),
                                   torch.tensor(sections, device=dev))
    angle = s["positions"].float()[:, :, axis] * s["inv_freq"]
    cos, sin = angle.cos()[:, :, None], angle.sin()[:, :, None]
    low, high = _pairs(case, sections, dev)

    def turn(x):
        xf = x.float()
        a, b = xf[..., low], xf[..., high]
        y = torch.empty_like(xf)
        y[..., low], y[..., high] = a * cos - b * sin, b * cos + a * sin
        return y.to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _allowed(s, lq, lk):
    """(B, Lq, Lk): whether a query sees a key; None where all do."""
    case, dev = s["case"], s["q"].device
    if not case["causal"] and not case["ragged"]:
        return None, None, None
    b = case["batch"]
    ql = s["q_lens"] if case["ragged"] else torch.full((b,), lq, device=dev)
    kl = s["kv_lens"] if case["ragged"] else torch.full((b,), lk, device=dev)
    i, j = torch.arange(lq, device=dev)[:, None], torch.arange(lk, device=dev)
    rows, keys = i < ql[:, None, None], j < kl[:, None, None]
    ok = rows & keys
    if case["causal"]:
        ok = ok & (j <= i + (kl - ql)[:, None, None])
    return ok, rows[:, :, 0], keys[:, 0]


def _plain_attention(s):
    case, T = s["case"], s["q"].dtype
    b, lq, hq, d = s["q"].shape
    lk, hk = s["k"].shape[1:3]
    g = hq // hk
    ok, rows, keys = _allowed(s, lq, lk)
    q = s["q"].float().view(b, lq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * lq, d)
    k = s["k"].float().transpose(1, 2)
    v = s["v"].float().transpose(1, 2)
    if ok is not None:  # what no query may see counts as zero, whatever it holds
        q = torch.where(rows[:, None, None, :].expand(b, 1, g, lq).reshape(b, 1, g * lq, 1), q, 0.0)
        k = torch.where(keys[:, None, :, None], k, 0.0)
        v = torch.where(keys[:, None, :, None], v, 0.0)
        hide = ~ok[:, None, None]
    scale = 1.0 / math.sqrt(d)

    def scores():
        x = torch.matmul(q, k.transpose(2, 3)).mul_(scale).view(b, hk, g, lq, lk)
        return x if ok is None else x.masked_fill_(hide, -math.inf)

    p = scores()
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = top + total.log()
    p = p.div_(torch.where(total == 0, 1.0, total)).view(b, hk, g * lq, lk)
    o = torch.matmul(p, v)

    def whole(x):  # back to (B, Lq, Hq, D)
        return x.view(b, hk, g, lq, d).permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d)

    out = {"out": whole(o).to(T), "lse": lse.view(b, hq, lq)}
    if case["direction"] == "train":
        do = s["dout"].float().view(b, lq, hk, g, d).permute(0, 2, 3, 1, 4)
        do = do.reshape(b, hk, g * lq, d)
        if ok is not None:
            do = torch.where(rows[:, None, None, :].expand(b, 1, g, lq).reshape(b, 1, g * lq, 1),
                             do, 0.0)
        dv = torch.matmul(p.transpose(2, 3), do)
        ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True))
        ds = ds.mul_(p).mul_(scale)
        out["dq"] = whole(torch.matmul(ds, k)).to(T)
        out["dk"] = torch.matmul(ds.transpose(2, 3), q).transpose(1, 2).to(T)
        out["dv"] = dv.transpose(1, 2).to(T)
    return out


# -------------------------------------------------------------------------------------- run

def _own_run(s):
    import activation_implicit_gemm_gb300 as fc
    case = s["case"]
    train = case["direction"] == "train"
    if case["op"] == "layer_norm":
        axis = 1
        if not train:
            return {"y": fc.layer_norm(s["x"], s["weight"], s["bias"], axis=axis, eps=1e-5)}
        y, mean, rstd = fc.layer_norm(s["x"], s["weight"], s["bias"], axis=axis, eps=1e-5,
                                      return_stats=True)
        dx, dw, db = fc.layer_norm_backward(s["dy"], s["x"], mean, rstd, s["weight"], s["bias"],
                                            axis=axis)
        return {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    if case["op"] == "rope":
        q, k = fc.rope(s["q"], s["k"], positions=s["positions"], inv_freq=s["inv_freq"],
                       sections=s["sections"], pairing=case["pairing"])
        return {"q": q, "k": k}
    mask = dict(causal=case["causal"], q_lens=s.get("q_lens"), kv_lens=s.get("kv_lens"))
    o, lse = fc.attention(s["q"], s["k"], s["v"], return_lse=True, **mask)
    out = {"out": o, "lse": lse}
    if train:
        out["dq"], out["dk"], out["dv"] = fc.attention_backward(
            s["dout"], s["q"], s["k"], s["v"], o, lse, **mask)
    return out


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "layer_norm":
        return _plain_norm(state)
    return _plain_rope(state) if op == "rope" else _plain_attention(state)


# ------------------------------------------------------------------------------------- work

def _seen(case):
    """Pairs of a query and a key that see each other, over the batch, for one head."""
    n = 0
    for q, k in zip(*_lens(case)):
        if not case["causal"]:
            n += q * k
            continue
        first = max(0, q - k)  # rows before it see nothing
        a, z = first + k - q + 1, k
        n += (a + z) * (q - first) // 2 if q > first else 0
    return n


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "layer_norm":
        n = case["outer"] * case["channels"] * case["inner"]
        p = case["channels"] * (4 if case["params"] == "f32" else 2)
        if case["direction"] == "train":  # x and dy in, y and dx out
            return {"bytes": 4 * n * e + 4 * p, "flops": 20 * n}
        return {"bytes": 2 * n * e + 2 * p, "flops": 8 * n}
    if case["op"] == "rope":
        tokens = case["batch"] * case["t"] * case["h"] * case["w"]
        n = tokens * (case["heads_q"] + case["heads_k"]) * case["dim"]
        axes = 3 if case["t"] > 1 else 2
        return {"bytes": 2 * n * e + 4 * tokens * axes + 4 * (case["dim"] // 2), "flops": 3 * n}
    hq, hk, d = case["heads_q"], case["heads_kv"], case["dim"]
    qs, ks = _lens(case)
    q, k = sum(qs) * hq * d, sum(ks) * hk * d
    whole_q = case["batch"] * case["len_q"] * hq
    pairs = _seen(case) * hq
    if case["direction"] == "train":  # q, dout in, out, dq out; k, v in, dk, dv out
        whole_k = case["batch"] * case["len_k"] * hk * d
        return {"bytes": e * (2 * q + 2 * whole_q * d + 2 * k + 2 * whole_k) + 4 * whole_q,
                "flops": 14 * pairs * d}
    return {"bytes": e * (q + whole_q * d + 2 * k) + 4 * whole_q, "flops": 4 * pairs * d}


# ------------------------------------------------------------------------------------ exact

def _exact_norm(s):
    case = s["case"]
    n, c, i = case["outer"], case["channels"], case["inner"]
    x = s["x"].double().view(n, c, i).transpose(1, 2).reshape(n * i, c)
    w, b = s["weight"].double(), s["bias"].double()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    sd = torch.sqrt(var + 1e-5)
    z = (x - mean) / sd

    def back(v):
        return v.view(n, i, c).transpose(1, 2).reshape(s["x"].shape)

    out = {"y": back(torch.addcmul(b, z, w))}
    if case["direction"] == "train":
        dy = s["dy"].double().view(n, c, i).transpose(1, 2).reshape(n * i, c)
        dz = dy * w
        along = torch.linalg.vecdot(dz, z).unsqueeze(1) / c
        out["dx"] = back((dz - dz.sum(1, keepdim=True) / c - z * along) / sd)
        out["dweight"] = torch.einsum("rc,rc->c", dy, z)
        out["dbias"] = torch.ones(1, n * i, dtype=dy.dtype, device=dy.device).matmul(dy)[0]
    return out


def _exact_rope(s):
    case, sections = s["case"], s["sections"]
    pos, freq = s["positions"].double(), s["inv_freq"].double()
    n = sum(sections)
    ends = [sum(sections[:a + 1]) for a in range(len(sections))]
    axis = [next(a for a, e in enumerate(ends) if p < e) for p in range(n)]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = torch.empty_like(x)
        for p in range(n):
            a = axis[p]
            start = ends[a] - sections[a]
            lo, hi = {"half": (p, p + n), "interleaved": (2 * p, 2 * p + 1),
                      "half_per_axis": (start + p, start + p + sections[a])}[case["pairing"]]
            turn = torch.polar(torch.ones_like(pos[..., a]), pos[..., a] * freq[p])
            z = torch.complex(x[..., lo], x[..., hi]) * turn[..., None]
            y[..., lo], y[..., hi] = z.real, z.imag
        out[name] = y
    return out


def _exact_attention(s):
    case = s["case"]
    B, Lq, H, D = s["q"].shape
    Lk, K = s["k"].shape[1:3]
    dev = s["q"].device
    qs, ks = _lens(case)
    f64 = dict(dtype=torch.float64, device=dev)
    out = torch.zeros(B, Lq, H, D, **f64)
    lse = torch.full((B, H, Lq), -math.inf, **f64)
    train = case["direction"] == "train"
    if train:
        dq = torch.zeros(B, Lq, H, D, **f64)
        dk, dv = torch.zeros(B, Lk, K, D, **f64), torch.zeros(B, Lk, K, D, **f64)
    for b in range(B):
        m, n = qs[b], ks[b]
        lead = max(0, m - n) if case["causal"] else 0  # rows that see nothing
        if n == 0 or m - lead <= 0:
            continue
        for h in range(H):
            kh = h // (H // K)
            q = s["q"][b, lead:m, h].double()
            k, v = s["k"][b, :n, kh].double(), s["v"][b, :n, kh].double()
            a = q @ k.T / math.sqrt(D)
            if case["causal"]:
                a = a + torch.full((m, n), -math.inf, **f64).triu(n - m + 1)[lead:]
            lse[b, h, lead:m] = torch.logsumexp(a, 1)
            a = (a - lse[b, h, lead:m, None]).exp()
            out[b, lead:m, h] = a @ v
            if train:
                g = s["dout"][b, lead:m, h].double()
                dv[b, :n, kh] += a.T @ g
                t = a * (g @ v.T - (g * out[b, lead:m, h]).sum(1, keepdim=True)) / math.sqrt(D)
                dq[b, lead:m, h] = t @ k
                dk[b, :n, kh] += t.T @ q
    got = {"out": out, "lse": lse}
    if train:
        got.update(dq=dq, dk=dk, dv=dv)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer_norm":
        return _exact_norm(s)
    if case["op"] == "rope":
        return _exact_rope(s)
    if work(case)["flops"] > 5e12:  # over about 20 seconds in 64 bits
        return None
    return _exact_attention(s)
