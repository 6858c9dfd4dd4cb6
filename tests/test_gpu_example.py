"""The vision-block example on the GPU: its gradients against a plain 64-bit block, and its
loss over a few steps."""
import importlib.util
import os

import pytest
import torch

from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "vision_block.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    spec = importlib.util.spec_from_file_location("vision_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    _ops.check_device()


def plain(p, images, heads):
    """The block's pooled features in 64 bits, from torch operations."""
    patch = p["patch"].shape[2]
    feat = torch.nn.functional.conv2d(images, p["patch"], stride=patch)
    n, c, rows, columns = feat.shape
    d = c // heads

    def norm(x, w, b):
        x = x - x.mean(-1, keepdim=True)
        return x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    def attend(q, k, v):
        s = torch.einsum("bihd,bjhd->bhij", q, k) * d ** -0.5
        return torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v)

    x = norm(feat.flatten(2).transpose(1, 2), p["stem_w"], p["stem_b"])
    h = norm(x, p["norm_w"], p["norm_b"])
    q, k, v = (h @ p["qkv"].t()).view(n, -1, 3, heads, d).unbind(2)
    first = d // 4
    sections = (first, d // 2 - first)
    freq = torch.cat([10000.0 ** -(torch.arange(m).double() / m) for m in sections])
    at = torch.cartesian_prod(torch.arange(rows), torch.arange(columns)).double()
    axis = torch.tensor([0] * sections[0] + [1] * sections[1])
    t = (at[:, axis] * freq)[:, None]

    def turn(u):
        lo, hi = u[..., :d // 2], u[..., d // 2:]
        return torch.cat([lo * t.cos() - hi * t.sin(), hi * t.cos() + lo * t.sin()], -1)

    y = x + attend(turn(q), turn(k), v).reshape(n, -1, c) @ p["proj"].t()
    keys = y.view(n, -1, heads, d)
    return attend(p["probe"].expand(n, 1, heads, d), keys, keys).reshape(n, c)


@pytest.mark.parametrize("n,height,width,c,heads,patch",
                         [(2, 64, 48, 128, 2, 16), (3, 40, 56, 96, 4, 8)])
def test_gradients(example, n, height, width, c, heads, patch):
    p = example.new_params(c, heads, patch, seed=3)
    g = torch.Generator().manual_seed(4)
    images = torch.randn(n, 3, height, width, generator=g).half()
    up = torch.randn(n, c, generator=g).half()
    pooled, kept = example.forward(p, images.cuda(), heads)
    grads = example.backward(p, kept, up.cuda())

    ref = {k: v.double().cpu().requires_grad_(k != "patch") for k, v in p.items()}
    want = plain(ref, images.double(), heads)
    want.backward(up.double())
    # some twenty tensors are rounded to f16 (2^-11 of each value) between the input and the
    # farthest gradient; in the 2-norm, with room for what softmax and norm add to each, 64 of them
    bound = 64 * 2.0 ** -11

    def far(a, b):
        return ((a.double().cpu() - b).norm() / b.norm()).item()

    assert far(pooled, want.detach()) < bound
    for name, grad in grads.items():
        assert far(grad, ref[name].grad) < bound, name


def test_loss_falls(example):
    p = example.new_params(64, 2, 8, seed=5)
    g = torch.Generator().manual_seed(6)
    images = torch.randn(4, 3, 32, 32, generator=g).half().cuda()
    target = torch.randn(4, 64, generator=g).cuda()
    losses = [example.step(p, images, target, 2, 2.0).item() for _ in range(10)]
    assert losses[-1] < losses[0]


def test_captured_in_a_graph(example):
    """The block's kernels (those that start beside their predecessor too) replayed from a CUDA
    graph on new inputs, against direct calls."""
    p = example.new_params(128, 2, 16, seed=7)
    g = torch.Generator().manual_seed(8)
    images = [torch.randn(3, 3, 64, 80, generator=g).half().cuda() for _ in range(3)]
    up = torch.randn(3, 128, generator=g).half().cuda()

    def run(x):
        pooled, kept = example.forward(p, x, 2)
        grads = example.backward(p, kept, up)
        return [pooled] + [grads[k] for k in sorted(grads)]

    x = images[0].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(3):
            run(x)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(x)
    for image in images:
        x.copy_(image)
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, run(image)):
            assert torch.equal(a, b)
