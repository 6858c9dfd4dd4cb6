"""One attention block of an image encoder, trained for a few steps.

The patch embedding is a FusedConv (stride == kernel; kept as it is, it has no gradient here).
Its channels-first features are normalised, become token rows, and go through

    h = layer_norm(x);  q, k, v = h Wqkv;  q, k turned by row and column;  y = x + attention Wo

and a learned query pools each image's tokens: a single query that all images share (its batch
stride is 0) over as many keys as the image has patches. Each operator's gradient runs back
through the same block; the matrix products between them are torch's.

    python examples/vision_block.py [--images 8] [--size 224] [--channels 768] [--heads 12]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_implicit_gemm_gb300 as fc  # noqa: E402


def new_params(channels, heads, patch, seed=0, device="cuda"):
    """Parameters in f16 as the block uses them, norms' in f32, and the positions' frequencies."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale):
        return (torch.randn(*shape, generator=g) * scale).half().to(device)

    c = channels
    return {
        "patch": normal(c, 3, patch, patch, scale=(3 * patch * patch) ** -0.5),
        "stem_w": torch.ones(c, device=device), "stem_b": torch.zeros(c, device=device),
        "norm_w": torch.ones(c, device=device), "norm_b": torch.zeros(c, device=device),
        "qkv": normal(3 * c, c, scale=c ** -0.5), "proj": normal(c, c, scale=c ** -0.5),
        "probe": normal(1, 1, heads, c // heads, scale=1.0),
        "freq": fc.rope_frequencies(sections(c // heads), device=device),
    }


def sections(head_dim):
    """The pairs of a head that turn by the row and by the column."""
    return (head_dim // 4, head_dim // 2 - head_dim // 4)


def grid_positions(rows, columns, device="cuda"):
    """(tokens, 2) int32: the row and column of each patch."""
    r = torch.arange(rows, dtype=torch.int32, device=device)
    c = torch.arange(columns, dtype=torch.int32, device=device)
    return torch.cartesian_prod(r, c).contiguous()


def forward(p, images, heads):
    """Pooled features (images, channels) and what the gradient needs."""
    patch = p["patch"].shape[2]
    feat = fc.fused_conv(images, p["patch"], strides=[patch, patch])
    n, c, rows, columns = feat.shape
    d = c // heads
    stem, s_mean, s_rstd = fc.layer_norm(feat, p["stem_w"], p["stem_b"], axis=1,
                                         return_stats=True)
    x = stem.flatten(2).transpose(1, 2).contiguous()
    h, mean, rstd = fc.layer_norm(x, p["norm_w"], p["norm_b"], return_stats=True)
    qkv = (h @ p["qkv"].t()).view(n, rows * columns, 3, heads, d)
    q, k, v = qkv.unbind(2)
    turn = {"positions": grid_positions(rows, columns, images.device),
            "inv_freq": p["freq"], "sections": sections(d)}
    fc.rope(q, k, **turn, out=q, k_out=k)
    a, lse = fc.attention(q, k, v, return_lse=True)
    y = x + a.view(n, -1, c) @ p["proj"].t()
    probe = p["probe"].expand(n, 1, heads, d)
    keys = y.view(n, -1, heads, d)
    pooled, pool_lse = fc.attention(probe, keys, keys, return_lse=True)
    kept = (feat, s_mean, s_rstd, x, h, mean, rstd, q, k, v, qkv, turn, a, lse, probe, keys,
            pooled, pool_lse)
    return pooled.reshape(n, c), kept


def backward(p, kept, dpooled):
    """Gradients of the parameters from the pooled features' gradient."""
    (feat, s_mean, s_rstd, x, h, mean, rstd, q, k, v, qkv, turn, a, lse, probe, keys, pooled,
     pool_lse) = kept
    n, tokens, c = x.shape
    g = {}
    dprobe, dk, dv = fc.attention_backward(dpooled.view(pooled.shape), probe, keys, keys, pooled,
                                           pool_lse)
    g["probe"] = dprobe.float().sum(0, keepdim=True)
    dy = (dk.float() + dv.float()).half().view(n, tokens, c)
    g["proj"] = dy.reshape(-1, c).t() @ a.reshape(-1, c)
    da = (dy @ p["proj"]).view(a.shape)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = dqkv.unbind(2)
    fc.attention_backward(da, q, k, v, a, lse, dq=dq, dk=dk, dv=dv)
    fc.rope(dq, dk, **turn, inverse=True, out=dq, k_out=dk)
    dqkv = dqkv.view(n, tokens, 3 * c)
    g["qkv"] = dqkv.reshape(-1, 3 * c).t() @ h.reshape(-1, c)
    dx, g["norm_w"], g["norm_b"] = fc.layer_norm_backward(dqkv @ p["qkv"], x, mean, rstd,
                                                          p["norm_w"], p["norm_b"])
    dstem = (dy + dx).transpose(1, 2).reshape(feat.shape).contiguous()
    _, g["stem_w"], g["stem_b"] = fc.layer_norm_backward(dstem, feat, s_mean, s_rstd,
                                                         p["stem_w"], p["stem_b"], axis=1)
    return g


def step(p, images, target, heads, rate):
    """One step of gradient descent on the mean squared distance to `target`; the loss before
    it. f16 gradients carry a factor of 2^10 until they are added."""
    pooled, kept = forward(p, images, heads)
    diff = pooled.float() - target
    grads = backward(p, kept, (diff * (1024.0 * 2.0 / diff.numel())).half())
    for name, grad in grads.items():
        p[name].copy_(p[name].float() - grad.float() * (rate / 1024.0))
    return diff.square().mean()


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--images", type=int, default=8)
    a.add_argument("--size", type=int, default=224)
    a.add_argument("--channels", type=int, default=768)
    a.add_argument("--heads", type=int, default=12)
    a.add_argument("--patch", type=int, default=16)
    a.add_argument("--steps", type=int, default=20)
    a.add_argument("--rate", type=float, default=2.0)
    a = a.parse_args()
    p = new_params(a.channels, a.heads, a.patch)
    g = torch.Generator(device="cuda").manual_seed(1)
    images = torch.randn(a.images, 3, a.size, a.size, generator=g, device="cuda").half()
    target = torch.randn(a.images, a.channels, generator=g, device="cuda")
    for i in range(a.steps):
        loss = step(p, images, target, a.heads, a.rate)
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}")


if __name__ == "__main__":
    main()
