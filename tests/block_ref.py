"""Plain 64-bit forms of the head norms with rotation and of the gated feed-forward block, with
error bounds derived from their arithmetic (CPU, small sizes). Symbols as in ops_ref: u is the
unit roundoff of a type, E32 that of f32."""
import torch

import ops_ref as R
from ops_ref import E32, TINY, U


# ------------------------------------------------------------------------------ head norms

def _turn(x, positions, inv_freq, sections, pairing, back=False):
    """(turned x, |u| + |v| of every element's pair) in 64 bits; elements without a pair stay."""
    y, size = x.clone(), torch.zeros_like(x)
    if positions is None:
        return y, size
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    for p, (lo, hi) in enumerate(R.rope_pairs(pairing, sections)):
        t = positions[..., axis[p]].double() * inv_freq[p].double()
        c, s = t.cos()[..., None], t.sin()[..., None] * (-1 if back else 1)
        a, b = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        size[..., lo] = size[..., hi] = a.abs() + b.abs()
    return y, size


# A turned pair: the kernel's angle is off by at most 2^-21, sine and cosine by 2 ulp, and the
# products and their sum round three times.
TURN = 2.0 ** -21 + 7 * E32


def _norm(x, eps):
    """(x in 64 bits, r, bound on r's relative error): a sum of D squares in any order is off by
    D + 1 roundings, halved by the root; mean, eps and rsqrt (2 ulp) count as six more."""
    xd = x.double()
    D = xd.shape[-1]
    r = 1.0 / torch.sqrt(xd.square().mean(-1, keepdim=True) + eps)
    return xd, r, ((D + 1) / 2 + 6) * E32


def norm_rope(x, w, positions, inv_freq, sections, pairing, eps):
    """(y, bound)."""
    T = x.dtype
    xd, r, er = _norm(x, eps)
    z = xd * r * (1.0 if w is None else w.double())
    y, size = _turn(z, positions, inv_freq, sections, pairing)
    tol = U[T] * y.abs() * 1.01 + (er + 2 * E32) * (size + z.abs()) + TURN * size + TINY[T]
    return y, tol


def norm_rope_backward(dy, x, w, positions, inv_freq, sections, pairing, eps):
    """{name: (gradient, bound)} for dx and, where there is a weight, dw."""
    T = x.dtype
    xd, r, er = _norm(x, eps)
    D = xd.shape[-1]
    wd = torch.ones(D).double() if w is None else w.double()
    g, size = _turn(dy.double(), positions, inv_freq, sections, pairing, back=True)
    eg = TURN * size
    a, ea = g * wd, eg * wd.abs() + E32 * (g * wd).abs()
    n = xd * r
    dot = (a * xd).sum(-1, keepdim=True)
    edot = (ea * xd.abs() + (D + 2) * E32 * (a * xd).abs()).sum(-1, keepdim=True)
    along, ealong = dot / D * r * r, (edot + dot.abs() * (2 * er + 4 * E32)) / D * r * r
    dx = r * (a - xd * along)
    tol = r * (ea + xd.abs() * ealong) + (er + 4 * E32) * r * (a.abs() + (xd * along).abs())
    out = {"dx": (dx, U[T] * dx.abs() * 1.01 + tol * 1.01 + TINY[T])}
    if w is not None:
        rows = g.numel() // D
        flat = lambda v: v.reshape(-1, D)  # noqa: E731
        dw = flat(g * n).sum(0)
        err = flat(eg * n.abs() + (er + (rows + 64) * E32) * (g * n).abs()).sum(0)
        out["dw"] = (dw, U[w.dtype] * dw.abs() * 1.01 + err * 1.01 + TINY[w.dtype])
    return out


# ------------------------------------------------------------------------ feed-forward block

def act(kind, v, alpha=1.702):
    """(act(v), its slope) in 64 bits."""
    if kind == "Silu":
        kind, alpha = "QuickGelu", 1.0
    if kind is None:
        return v, torch.ones_like(v)
    if kind == "Relu":
        return v.clamp(min=0.0), (v > 0).double()
    if kind == "Sigmoid":
        p = torch.sigmoid(v)
        return p, p * torch.sigmoid(-v)
    if kind == "QuickGelu":
        p = torch.sigmoid(alpha * v)
        return v * p, p * (1.0 + alpha * v * (1.0 - p))
    if kind == "Gelu":
        p = 0.5 * torch.erfc(-v * 0.5 ** 0.5)
        return v * p, p + v * (-0.5 * v * v).exp() * (0.5 / torch.pi) ** 0.5
    k, c = (2.0 / torch.pi) ** 0.5, 0.044715
    t = torch.tanh(k * (v + c * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * c * v * v)


def _product(a, ea, b, K):
    """(a b^T, bound): the operands' errors through the product, and a sum of K products. On the
    tensor instructions each addition may cut instead of round (2 E32 of the sum of magnitudes);
    split f32 operands drop at most 12 E32 of a product, and joins of partial sums count 20."""
    size = a.abs() @ b.abs().t()
    return a @ b.t(), ea @ b.abs().t() + (2 * K + 32) * E32 * size


def gated_mlp(x, wg, wu, wd, bg=None, bu=None, bd=None, activation="Silu", alpha=1.702, dy=None):
    """{name: (value, bound)}: y, and with dy the gradients. h, dg and du are rounded to x's type
    as operands of the products that follow."""
    T, u = x.dtype, U[x.dtype]
    op = 0.0 if T == torch.float32 else u * 1.01  # of an operand
    tiny = TINY[T]
    X, G, UP, D = (t.double() for t in (x, wg, wu, wd))
    n, c = X.shape
    f, o = G.shape[0], D.shape[0]
    vec = lambda b, m: torch.zeros(m).double() if b is None else b.double()  # noqa: E731
    none = torch.zeros_like(X)
    g, eg = _product(X, none, G, c)
    v, ev = _product(X, none, UP, c)
    g, v = g + vec(bg, f), v + vec(bu, f)
    eg, ev = eg + 2 * E32 * (g.abs() + vec(bg, f).abs()), ev + 2 * E32 * (v.abs() + vec(bu, f).abs())
    a, s = act(activation, g, alpha)
    lip = 1.2 * max(1.0, alpha if activation == "QuickGelu" else 1.0)
    # slopes of act stay under lip, those of its slope too; the functions themselves are within
    # a few ulp of arguments that are rounded (exp of g^2, say, turns that into g^2 ulp)
    ea = lip * eg + (16 + 2 * g * g) * E32 * a.abs() + 8 * E32 * g.abs() + 8 * E32
    if activation == "Relu":
        es = (g.abs() <= eg).double()
    elif activation is None:
        ea, es = eg, torch.zeros_like(g)
    else:
        es = lip * lip * eg + 64 * E32 * (1 + g.abs() ** 3)
    h = a * v
    eh = ea * v.abs() + (a.abs() + ea) * ev + 2 * E32 * h.abs()
    eh = eh + op * (h.abs() + eh) + tiny
    y, ey = _product(h, eh, D, f)
    y = y + vec(bd, o)
    out = {"y": (y, u * y.abs() * 1.01 + ey * 1.01 + 2 * E32 * vec(bd, o).abs() + tiny)}
    if dy is None:
        return out
    dyd = dy.double()
    dh, edh = _product(dyd, torch.zeros_like(dyd), D.t(), o)

    def rounded(val, err):
        err = err + 4 * E32 * val.abs()
        return err + op * (val.abs() + err) + tiny

    dg, du = dh * v * s, dh * a
    edg = rounded(dg, edh * (v.abs() + ev) * (s.abs() + es)
                  + dh.abs() * (ev * (s.abs() + es) + v.abs() * es))
    edu = rounded(du, edh * (a.abs() + ea) + dh.abs() * ea)
    both = torch.cat([G.t(), UP.t()], 1)
    dx, edx = _product(torch.cat([dg, du], 1), torch.cat([edg, edu], 1), both, 2 * f)
    last = lambda t, e: (t, u * t.abs() * 1.01 + e * 1.01 + tiny)  # noqa: E731
    out["dx"] = last(dx, edx)
    out["dw_gate"] = last(*_product(dg.t(), edg.t(), X.t(), n))
    out["dw_up"] = last(*_product(du.t(), edu.t(), X.t(), n))
    dwd, ed = _product(h.t(), eh.t(), dyd.t(), n)
    out["dw_down"] = last(dwd.t(), ed.t())
    for name, b, val, err in (("db_gate", bg, dg, edg), ("db_up", bu, du, edu),
                              ("db_down", bd, dyd, torch.zeros_like(dyd))):
        if b is not None:
            out[name] = last(val.sum(0), err.sum(0) + (n + 32) * E32 * val.abs().sum(0))
    return out
