"""The encoder-block example on the GPU: layer norm, head norms with rotation, attention and the
gated feed-forward block together, forward and back, against a plain 64-bit block; captured in a
graph; one step run."""
import importlib.util
import os

import pytest
import torch

from activation_implicit_gemm_gb300 import _build, _ops

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "encoder_block.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    spec = importlib.util.spec_from_file_location("encoder_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    _ops.check_device()


def plain(p, x, positions, heads):
    """The block's output in 64 bits, from torch operations."""
    n, t, c = x.shape
    d = c // heads

    def layer_norm(v, w, b):
        v = v - v.mean(-1, keepdim=True)
        return v / (v.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    def turn(v, w):
        v = v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        first = d // 4
        axis = torch.tensor([0] * first + [1] * (d // 2 - first))
        angle = (positions.double()[:, axis] * p["freq"])[:, None]
        lo, hi = v[..., :d // 2], v[..., d // 2:]
        return torch.cat([lo * angle.cos() - hi * angle.sin(),
                          hi * angle.cos() + lo * angle.sin()], -1)

    h = layer_norm(x, p["norm1_w"], p["norm1_b"])
    q, k, v = (h @ p["qkv"].t()).view(n, t, 3, heads, d).unbind(2)
    s = torch.einsum("bihd,bjhd->bhij", turn(q, p["q_norm"]), turn(k, p["k_norm"])) * d ** -0.5
    a = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v).reshape(n, t, c)
    y = x + a @ p["proj"].t()
    h = layer_norm(y, p["norm2_w"], p["norm2_b"])
    g, u = (h @ p["gate_up"].t() + p["gate_up_b"]).chunk(2, -1)
    return y + (g * torch.sigmoid(g) * u) @ p["down"].t() + p["down_b"]


@pytest.mark.parametrize("dtype,u", [(torch.float32, 2.0 ** -24), (torch.float16, 2.0 ** -11),
                                     (torch.bfloat16, 2.0 ** -8)])
@pytest.mark.parametrize("n,rows,columns,c,heads,hidden",
                         [(2, 5, 7, 128, 2, 200), (3, 12, 11, 96, 3, 264)])
def test_gradients(example, n, rows, columns, c, heads, hidden, dtype, u):
    torch.backends.cuda.matmul.allow_tf32 = False
    p = example.new_params(c, heads, hidden, dtype, seed=3)
    g = torch.Generator().manual_seed(4)
    x, up = (torch.randn(n, rows * columns, c, generator=g).to(dtype) for _ in range(2))
    positions = example.grid_positions(rows, columns)
    z, kept = example.forward(p, x.cuda(), positions, heads)
    dx, grads = example.backward(p, kept, up.cuda())

    ref = {k: v.double().cpu().requires_grad_(k != "freq") for k, v in p.items()}
    xd = x.double().requires_grad_()
    want = plain(ref, xd, positions.cpu(), heads)
    want.backward(up.double())
    # some thirty tensors are rounded to the type (u of each value) between the input and the
    # farthest gradient, and each of the five sums over rows or channels in f32 adds a few u of
    # f32; in the 2-norm, with room for what softmax and norms add to each, 64 of them
    bound = 64 * u

    def far(a, b):
        return ((a.double().cpu() - b).norm() / b.norm()).item()

    assert far(z, want.detach()) < bound
    assert far(dx, xd.grad) < bound
    assert set(grads) == set(p) - {"freq"}
    for name, grad in grads.items():
        assert far(grad, ref[name].grad) < bound, name


def test_a_step_runs(example):
    p = example.new_params(64, 2, 96, seed=5)
    g = torch.Generator().manual_seed(6)
    x = torch.randn(4, 12, 64, generator=g).bfloat16().cuda()
    target = torch.randn(4, 12, 64, generator=g).cuda()
    before = {k: v.clone() for k, v in p.items()}
    loss = example.step(p, x, target, example.grid_positions(3, 4), 2, 1.0)
    assert torch.isfinite(loss)
    for name, v in p.items():
        assert torch.isfinite(v).all()
        assert name == "freq" or not torch.equal(v, before[name]), name


def test_captured_in_a_graph(example):
    """The block replayed from a CUDA graph on new inputs, against direct calls, while an eager
    step of the same parameters lives."""
    p = example.new_params(128, 2, 200, seed=7)
    g = torch.Generator().manual_seed(8)
    xs = [torch.randn(3, 35, 128, generator=g).bfloat16().cuda() for _ in range(3)]
    up = torch.randn(3, 35, 128, generator=g).bfloat16().cuda()
    positions = example.grid_positions(5, 7)

    def run(x):
        z, kept = example.forward(p, x, positions, 2)
        dx, grads = example.backward(p, kept, up)
        return [z, dx] + [grads[k] for k in sorted(grads)]

    x = xs[0].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(3):
            run(x)
    torch.cuda.current_stream().wait_stream(stream)
    eager = run(xs[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(x)
    for v in xs:
        x.copy_(v)
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, run(v)):
            assert torch.equal(a, b)
    for a, b in zip(eager, run(xs[1])):
        assert torch.equal(a, b)
