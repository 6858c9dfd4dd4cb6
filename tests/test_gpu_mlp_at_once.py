"""Calls of the block's operators at once: from several threads on streams of their own, in two graphs
replayed beside each other, and two backward passes of one forward pass. All give the bits of calls
that run alone."""
import random
import threading

import pytest
import torch

import ops_ref as R
import activation_implicit_gemm_gb300 as fc
from activation_implicit_gemm_gb300 import _build, _ops
from test_gpu_mlp import case

pytestmark = pytest.mark.gpu

SIZES = [(700, 520, 1030, 264, "f32"), (2600, 1031, 1104, 1048, "f16"), (5, 768, 2048, 768, "bf16"),
         (300, 256, 512, 256, "bf16"), (20, 333, 777, 100, "f16"), (40000, 64, 96, 64, "f16")]


@pytest.fixture(scope="module", autouse=True)
def cuda_lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    _build.build()
    yield
    _ops.check_device()


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.fixture(scope="module")
def runs():
    """Calls of different sizes, and what each gives alone."""
    def mlp(seed, n, c, f, o, dtype):
        x, wg, wu, wd, b, dy = case(seed, n, c, f, o, R.TYPES[dtype])
        dev = [t.cuda() for t in (x, wg, wu, wd)]
        dy, how = dy.cuda(), {k: t.cuda() for k, t in zip(("b_gate", "b_up", "b_down"), b)}

        def run():
            y, saved = fc.gated_mlp(*dev, **how, return_saved=True)
            first = fc.gated_mlp_backward(dy, *dev, saved, **how)
            second = fc.gated_mlp_backward(dy, *dev, saved, **how)
            return [y, *first, *second]
        return run

    def heads(seed, n):
        q, dq = (R.normal(seed + i, (2, n, 8, 64), torch.bfloat16).cuda() for i in range(2))
        w = R.normal(seed + 2, (64,), torch.bfloat16).cuda()

        def run():
            return [fc.norm_rope(q, weight=w), *fc.norm_rope_backward(dq, q, weight=w)[::2]]
        return run

    calls = [mlp(500 + i, *s) for i, s in enumerate(SIZES)] + [heads(600, 7), heads(700, 3000)]
    want = [call() for call in calls]
    for out in want[:len(SIZES)]:
        assert same(out[1:8], out[8:])
    return calls, want


def test_threads_with_streams_of_their_own(runs):
    calls, want = runs
    bad = []

    def work(seed):
        rng, stream = random.Random(seed), torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                i = rng.randrange(len(calls))
                if not same(calls[i](), want[i]):
                    bad.append((seed, i))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_two_graphs_beside_each_other(runs):
    calls, want = runs
    graphs = []
    for i in (1, 5, 0, 7):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = calls[i]()
        graphs.append((torch.cuda.Stream(), graph, out, want[i]))
    for _ in range(5):
        for stream, graph, _, _ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(same(out, ref) for _, _, out, ref in graphs)
