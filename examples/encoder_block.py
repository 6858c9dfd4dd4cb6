"""A whole encoder block over token rows, trained for a few steps.

    h = layer_norm(x);  q, k, v = h Wqkv;  q, k = norm_rope(q, k)
    y = x + attention(q, k, v) Wo
    z = y + gated_mlp(layer_norm(y))

Queries and keys are normalised head by head and turned by row and column in one pass. Each
operator's gradient runs back through the same block; the matrix products between them are
torch's.

    python examples/encoder_block.py [--images 8] [--rows 14] [--columns 14] [--channels 768]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_implicit_gemm_gb300 as fc  # noqa: E402


def new_params(channels, heads, hidden, dtype=torch.bfloat16, seed=0, device="cuda"):
    """Parameters as the block uses them, norms' in f32, and the positions' frequencies."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale, shift=0.0, to=dtype):
        return (torch.randn(*shape, generator=g) * scale + shift).to(to).to(device)

    c, d, f32 = channels, channels // heads, torch.float32
    return {
        "norm1_w": torch.ones(c, device=device), "norm1_b": torch.zeros(c, device=device),
        "norm2_w": torch.ones(c, device=device), "norm2_b": torch.zeros(c, device=device),
        "qkv": normal(3 * c, c, scale=c ** -0.5), "proj": normal(c, c, scale=c ** -0.5),
        "q_norm": normal(d, scale=0.1, shift=1.0, to=f32),
        "k_norm": normal(d, scale=0.1, shift=1.0, to=f32),
        "gate_up": normal(2 * hidden, c, scale=c ** -0.5),  # one packed weight
        "gate_up_b": normal(2 * hidden, scale=0.02),
        "down": normal(c, hidden, scale=hidden ** -0.5), "down_b": normal(c, scale=0.02),
        "freq": fc.rope_frequencies(sections(d), device=device),
    }


def sections(head_dim):
    """The pairs of a head that turn by the row and by the column."""
    return (head_dim // 4, head_dim // 2 - head_dim // 4)


def grid_positions(rows, columns, device="cuda"):
    """(tokens, 2) int32: the row and column of each token."""
    r = torch.arange(rows, dtype=torch.int32, device=device)
    c = torch.arange(columns, dtype=torch.int32, device=device)
    return torch.cartesian_prod(r, c).contiguous()


def _heads_args(p, positions):
    return {"weight": p["q_norm"], "k_weight": p["k_norm"], "positions": positions,
            "inv_freq": p["freq"], "sections": sections(2 * p["freq"].numel())}


def _mlp_args(p):
    f = p["down"].shape[1]
    return ((p["gate_up"][:f], p["gate_up"][f:], p["down"]),
            {"b_gate": p["gate_up_b"][:f], "b_up": p["gate_up_b"][f:], "b_down": p["down_b"]})


def forward(p, x, positions, heads):
    """The block's output for x (batch, tokens, channels), and what the gradient needs."""
    n, t, c = x.shape
    h1, mean1, rstd1 = fc.layer_norm(x, p["norm1_w"], p["norm1_b"], return_stats=True)
    qkv = (h1 @ p["qkv"].t()).view(n, t, 3, heads, c // heads)
    q0, k0, v = qkv.unbind(2)
    q, k = fc.norm_rope(q0, k0, **_heads_args(p, positions))
    a, lse = fc.attention(q, k, v, return_lse=True)
    y = x + a.view(n, t, c) @ p["proj"].t()
    h2, mean2, rstd2 = fc.layer_norm(y, p["norm2_w"], p["norm2_b"], return_stats=True)
    weights, biases = _mlp_args(p)
    m, saved = fc.gated_mlp(h2, *weights, **biases, return_saved=True)
    kept = (x, h1, mean1, rstd1, q0, k0, v, q, k, a, lse, y, h2, mean2, rstd2, saved, positions)
    return y + m, kept


def backward(p, kept, dz):
    """Gradients of x and of the parameters from the output's gradient."""
    x, h1, mean1, rstd1, q0, k0, v, q, k, a, lse, y, h2, mean2, rstd2, saved, positions = kept
    n, t, c = x.shape
    g = {}
    weights, biases = _mlp_args(p)
    dh2, dgate, dup, g["down"], dbg, dbu, g["down_b"] = fc.gated_mlp_backward(
        dz, h2, *weights, saved, **biases)
    g["gate_up"], g["gate_up_b"] = torch.cat([dgate, dup]), torch.cat([dbg, dbu])
    dy, g["norm2_w"], g["norm2_b"] = fc.layer_norm_backward(dh2, y, mean2, rstd2, p["norm2_w"],
                                                            p["norm2_b"])
    dy = dy + dz
    g["proj"] = dy.reshape(-1, c).t() @ a.reshape(-1, c)
    da = (dy @ p["proj"]).view(a.shape)
    dqkv = torch.empty(n, t, 3, *a.shape[2:], dtype=x.dtype, device=x.device)
    dq, dk, dv = dqkv.unbind(2)
    fc.attention_backward(da, q, k, v, a, lse, dq=dq, dk=dk, dv=dv)
    _, _, g["q_norm"], g["k_norm"] = fc.norm_rope_backward(
        dq, q0, dk, k0, **_heads_args(p, positions), dq=dq, dk=dk)
    dqkv = dqkv.view(-1, 3 * c)
    g["qkv"] = dqkv.t() @ h1.reshape(-1, c)
    dx, g["norm1_w"], g["norm1_b"] = fc.layer_norm_backward(
        (dqkv @ p["qkv"]).view(x.shape), x, mean1, rstd1, p["norm1_w"], p["norm1_b"])
    return dx + dy, g


def step(p, x, target, positions, heads, rate):
    """One step of gradient descent on the mean squared distance to `target`; the loss before it."""
    z, kept = forward(p, x, positions, heads)
    diff = z.float() - target
    _, grads = backward(p, kept, (diff * (2.0 / diff.numel())).to(x.dtype))
    for name, grad in grads.items():
        p[name].copy_(p[name].float() - grad.float() * rate)
    return diff.square().mean()


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--images", type=int, default=8)
    a.add_argument("--rows", type=int, default=14)
    a.add_argument("--columns", type=int, default=14)
    a.add_argument("--channels", type=int, default=768)
    a.add_argument("--heads", type=int, default=12)
    a.add_argument("--hidden", type=int, default=2048)
    a.add_argument("--steps", type=int, default=20)
    a.add_argument("--rate", type=float, default=20.0)
    a = a.parse_args()
    p = new_params(a.channels, a.heads, a.hidden)
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = (a.images, a.rows * a.columns, a.channels)
    x = torch.randn(*shape, generator=g, device="cuda").bfloat16()
    target = torch.randn(*shape, generator=g, device="cuda")
    positions = grid_positions(a.rows, a.columns)
    for i in range(a.steps):
        loss = step(p, x, target, positions, a.heads, a.rate)
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}")


if __name__ == "__main__":
    main()
