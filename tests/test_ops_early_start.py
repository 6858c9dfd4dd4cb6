"""attn_mma_dq and attn_tc_dq start beside the kernel launched before them and read their inputs
before they wait for it, so every such read must come from L2: nothing orders the L1 of their SM.
The reads are checked in the source (no GPU); on the GPU, passes that follow each other over the
same buffers give the bits of passes that run alone."""
import os
import re

import pytest
import torch

import ops_ref as R

OPS = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "activation_implicit_gemm_gb300", "csrc", "ops")


def source(*path):
    text = open(os.path.join(OPS, *path)).read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, name):
    """The braces that follow the definition of `name`."""
    start = text.index("{", text.index(name + "("))
    depth = 0
    for at in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        if depth == 0:
            return text[start:at + 1]
    raise AssertionError(name)


def test_tiles_are_read_from_l2():
    load = body(source("attn_geom.cuh"), "load_tile")
    copies = set(re.findall(r"cp_async\d+\w*(?=\()", load))
    assert copies and "__ldcg(" in load
    ptx = source(os.pardir, "ptx.cuh")
    for name in copies:
        assert "cp.async.cg." in body(ptx, name), name
    assert "__ldcg(g.q_lens" in source("attn_geom.cuh")


@pytest.mark.parametrize("file,kernel,early", [("attn_mma.cuh", "attn_mma_dq", ("lse", "delta")),
                                               ("k_attn_tc_bwd.cu", "attn_tc_dq", ("stat",))])
def test_statistics_are_read_from_l2(file, kernel, early):
    text = body(source(file), kernel)
    assert text.index("ptx::pdl_wait") > text.index("__ldcg(")  # the wait comes late
    for name in early:
        reads = [m.start() for m in re.finditer(rf"(?<![\w.]){name}(\[| \+ )", text)]
        assert reads
        for at in reads:
            assert text[:at].endswith("__ldcg("), (kernel, text[at - 20:at + 20])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [("f32", 72), ("f32", 33), ("f16", 64), ("bf16", 128)])
def test_passes_that_follow_each_other(dtype, D):
    """The inputs are written in place right before each pass, and passes are not waited for."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import activation_implicit_gemm_gb300 as fc
    T = R.TYPES[dtype]
    B, L, H, K = 2, 300, 6, 2
    kl = torch.tensor([300, 171], dtype=torch.int32).cuda()
    sets = [[R.normal(40 + 4 * i + j, (B, L, h, D), T).cuda()
             for j, h in enumerate((H, K, K, H))] for i in range(3)]

    def run(q, k, v, g):
        out, lse = fc.attention(q, k, v, causal=True, kv_lens=kl, return_lse=True)
        return (out, *fc.attention_backward(g, q, k, v, out, lse, causal=True, kv_lens=kl))

    want = []
    for s in sets:
        want.append(run(*s))
        torch.cuda.synchronize()
    buffers = [t.clone() for t in sets[0]]
    got = []
    for n in range(30):
        for b, t in zip(buffers, sets[n % 3]):
            b.copy_(t)
        got.append(run(*buffers))
    torch.cuda.synchronize()
    for n, outs in enumerate(got):
        for a, b in zip(outs, want[n % 3]):
            assert torch.equal(a, b), n
