"""Plain 64-bit forms of the token-side operators and error bounds derived from their
arithmetic, for the parity tests (CPU, small sizes).

u is the unit roundoff of a type: 2^-24 (f32), 2^-11 (f16), 2^-8 (bf16). The kernels sum in
f32 and round each output once; on tensor cores the probabilities and score gradients are
also rounded to the element type before their products.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
E32 = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def normal(seed, shape, dtype, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale + shift).to(dtype)


def check(got, ref, tol, what):
    """|got - ref| <= tol element by element; infinities must be equal."""
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    same = got == ref
    bad = ~(same | ((got - ref).abs() <= tol))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        t = tol[i] if torch.is_tensor(tol) and tol.dim() else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, first "
                             f"{i}: {got[i].item()!r} against {ref[i].item()!r}, tol {float(t):.3e}")


# ---------------------------------------------------------------------------- layer norm

def layer_norm(x, w, b, axis, eps):
    """(y, mean, rstd, bound on y's error) in 64 bits."""
    T = x.dtype
    xd = x.double().movedim(axis, -1)
    C = xd.shape[-1]
    mean = xd.mean(-1)
    var = (xd - mean[..., None]).square().mean(-1)
    rstd = 1.0 / torch.sqrt(var + eps)
    xhat = (xd - mean[..., None]) * rstd[..., None]
    wd = torch.ones(C).double() if w is None else w.double()
    bd = torch.zeros(C).double() if b is None else b.double()
    y = xhat * wd + bd
    e = norm_error(xd, rstd)
    tol = U[T] * y.abs() + e[..., None] * wd.abs() * (1 + xhat.abs()) + 4 * E32 * bd.abs()
    tol = tol * 1.01 + TINY[T]
    return y.movedim(-1, axis), mean, rstd, tol.movedim(-1, axis)


def norm_error(xd, rstd):
    """Bound on the error of xhat over 1 + |xhat|: the f32 sums run over at most C / 32 terms in
    sequence and a tree of 10 levels, each adding 2^-24 of the largest |x| in units of the
    deviation; the handful of roundings after them counts as 16 more."""
    C = xd.shape[-1]
    return (C / 32 + 32) * E32 * (1 + xd.abs().amax(-1) * rstd)


def layer_norm_backward(dy, x, w, b, axis, eps):
    """{name: (gradient, bound)} in 64 bits."""
    T = x.dtype
    xd, dyd = x.double().movedim(axis, -1), dy.double().movedim(axis, -1)
    C = xd.shape[-1]
    mean = xd.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((xd - mean).square().mean(-1, keepdim=True) + eps)
    h = (xd - mean) * rstd
    g = dyd if w is None else dyd * w.double()
    m1, m2 = g.mean(-1, keepdim=True), (g * h).mean(-1, keepdim=True)
    dx = rstd * (g - m1 - h * m2)
    e = norm_error(xd, rstd[..., 0])[..., None]
    a1, a2 = g.abs().mean(-1, keepdim=True), (g * h).abs().mean(-1, keepdim=True)
    spread = g.abs().mean(-1, keepdim=True) + (g.abs() * (1 + h.abs())).mean(-1, keepdim=True)
    tol = rstd * e * (g.abs() + a1 + h.abs() * a2 + (1 + h.abs()) * (a2 + spread) + spread)
    out = {"dx": (dx.movedim(-1, axis), (U[T] * dx.abs() + tol * 1.01 + TINY[T]).movedim(-1, axis))}
    rows = dyd.reshape(-1, C)
    N = rows.shape[0]
    hr, er = h.reshape(-1, C), e.expand_as(h).reshape(-1, C)
    n32 = (N / 32 + 512) * E32  # sums over rows: sequences of N / 32 at most, joined in order
    if w is not None:
        t = (rows * hr).sum(0)
        out["dweight"] = (t, U[w.dtype] * t.abs() * 1.01 + n32 * (rows * hr).abs().sum(0)
                          + (er * rows.abs() * (1 + hr.abs())).sum(0) + TINY[w.dtype])
    if b is not None:
        s = rows.sum(0)
        out["dbias"] = (s, U[b.dtype] * s.abs() * 1.01 + n32 * rows.abs().sum(0) + TINY[b.dtype])
    return out


# ------------------------------------------------------------------------------ positions

def rope_pairs(pairing, sections):
    n = sum(sections)
    pairs, start = [], 0
    for size in sections:
        for i in range(size):
            p = start + i
            pairs.append({"interleaved": (2 * p, 2 * p + 1), "half": (p, p + n),
                          "half_per_axis": (start + p, start + p + size)}[pairing])
        start += size
    return pairs


def rope(x, positions, inv_freq, sections, pairing, inverse=False):
    """(turned x, bound): angles in 64 bits from the f32 frequencies. The kernel's reduced angle
    is off by at most 2^-21 (half an ulp of an angle below 4 twice, and the product's and the
    reduction's remainders) and sine and cosine by 2 ulp."""
    xd, T = x.double(), x.dtype
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    y = xd.clone()
    tol = torch.zeros_like(xd)
    for p, (lo, hi) in enumerate(rope_pairs(pairing, sections)):
        t = positions[..., axis[p]].double() * inv_freq[p].double()
        c, s = t.cos()[..., None], t.sin()[..., None]
        if inverse:
            s = -s
        u, v = xd[..., lo], xd[..., hi]
        y[..., lo], y[..., hi] = u * c - v * s, v * c + u * s
        size = (u.abs() + v.abs()) * (2.0 ** -21 + 4 * E32)
        tol[..., lo], tol[..., hi] = size, size
    return y, U[T] * y.abs() * 1.01 + tol + TINY[T]


# ------------------------------------------------------------------------------ attention

def allowed(B, Lq, Lk, causal, q_lens, kv_lens):
    """(B, Lq, Lk) bool: whether a query sees a key."""
    ql = torch.full((B,), Lq) if q_lens is None else q_lens.long().clamp(0, Lq)
    kl = torch.full((B,), Lk) if kv_lens is None else kv_lens.long().clamp(0, Lk)
    i, j = torch.arange(Lq)[:, None], torch.arange(Lk)
    ok = (i < ql[:, None, None]) & (j < kl[:, None, None])
    if causal:
        ok = ok & (j <= i + (kl - ql)[:, None, None])
    return ok


def _rows(x):  # (B, L, H, D) -> (B, H, L, D)
    return x.double().transpose(1, 2)


def attention(q, k, v, *, causal=False, scale=None, q_lens=None, kv_lens=None, dout=None):
    """{name: (value, bound)} in 64 bits: out and lse, and with dout the gradients."""
    T, u = q.dtype, U[q.dtype]
    B, Lq, H, D = q.shape
    Lk, K = k.shape[1:3]
    G = H // K
    scale = D ** -0.5 if scale is None else scale
    ok = allowed(B, Lq, Lk, causal, q_lens, kv_lens)
    seen_q, seen_k = ok.any(2), ok.any(1)
    zero = torch.zeros((), dtype=torch.float64)
    # tokens that see nothing and are seen by nothing count as zero, whatever they hold
    qd = torch.where(seen_q[:, None, :, None], _rows(q), zero)
    kd = torch.where(seen_k[:, None, :, None], _rows(k), zero).repeat_interleave(G, 1)
    vd = torch.where(seen_k[:, None, :, None], _rows(v), zero).repeat_interleave(G, 1)
    ok = ok[:, None]
    s = torch.where(ok, qd @ kd.transpose(2, 3) * scale, torch.full((), -math.inf).double())
    top = s.amax(-1, keepdim=True) if Lk else torch.full((B, H, Lq, 1), -math.inf).double()
    safe = torch.where(top == -math.inf, zero, top)
    e = (s - safe).exp()
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, torch.ones_like(total), total)
    o = p @ vd
    lse = (safe + total.log())[..., 0]
    # a probability's relative error: the f32 score (a sum of D products, in sequence at worst),
    # its exponential (a few ulp, and the f32 product with log2 e of scores up to |s|), the sum
    # of up to Lk terms and, rounded for the tensor cores, u
    size = (qd.abs() @ kd.abs().transpose(2, 3) * scale).amax(-1, keepdim=True) if Lk else zero
    ep = (2 * D + 8) * E32 * size + (Lk + 32) * E32 + 2.0 ** -20
    rp = ep + (u if T != torch.float32 else 0.0)
    tiny = TINY[T] * 2
    ap = p @ vd.abs()
    to = u * o.abs() * 1.01 + rp * ap + tiny * (1 + vd.abs().sum(2, keepdim=True))
    back = lambda x: x.transpose(1, 2)  # noqa: E731
    res = {"out": (back(o), back(to)),
           "lse": (lse, torch.nan_to_num((ep[..., 0] if Lk else zero) + 4 * E32 * lse.abs(), posinf=0.0)
                   + 4 * E32)}
    if dout is None:
        return res
    g = torch.where(seen_q[:, None, :, None], _rows(dout), zero)
    dp = g @ vd.transpose(2, 3)
    delta = (g * o).sum(-1, keepdim=True)
    ds = torch.where(ok, p * (dp - delta), zero)
    # delta comes from the rounded out; the products of dp are f32 sums
    ed = (u + rp) * (g.abs() * ap).sum(-1, keepdim=True) + (u if True else 0) * (
        g.abs() * o.abs()).sum(-1, keepdim=True)
    es = rp * ds.abs() + p * (ed + (D + 8) * E32 * (g.abs() @ vd.abs().transpose(2, 3))) + tiny
    es = torch.where(ok, es, zero)
    ts = lambda x: x.transpose(2, 3)  # noqa: E731
    share = lambda x: back(x.view(B, K, G, Lk, D).sum(2))  # noqa: E731
    n32 = lambda n: (n + 32) * E32  # noqa: E731
    dq, dk, dv = ds @ kd * scale, ts(ds) @ qd * scale, ts(p) @ g
    ads = ds.abs()
    tq = (es + n32(Lk) * ads) @ kd.abs() * scale
    tk = ts(es + n32(Lq * G) * ads) @ qd.abs() * scale
    tv = ts((rp + n32(Lq * G)) * p + tiny * ok) @ g.abs()
    res["dq"] = (back(dq), back(u * dq.abs() * 1.01 + tq + tiny))
    res["dk"] = (share(dk), u * share(dk).abs() * 1.01 + share(tk) + tiny)
    res["dv"] = (share(dv), u * share(dv).abs() * 1.01 + share(tv) + tiny)
    return res
