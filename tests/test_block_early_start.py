"""Kernels of the gated block that read before they wait for the launch before them: the second
product of few tokens reads its first weights, and the bias sums all they add. Such reads must come
from L2, since nothing orders the L1 of their SM, and the launch before them must have waited for
what they read. Checked in the source (no GPU); on the GPU, passes that follow each other over the
same buffers give the bits of passes that run alone (test_gpu_mlp)."""
import re

from test_ops_early_start import body, source


def test_first_weights_come_from_l2():
    text = source("k_mlp_few.cu")
    kernel = body(text, "mlp_few")
    wait = kernel.index("ptx::pdl_wait")
    early = kernel[:wait]
    calls = re.findall(r"load_weights\(([^)]*)\)", early)
    assert calls == ["first, true"]
    loads = body(text, "load_row")
    assert "if (HOW == kEarly) return __ldcg(" in loads
    assert "HOW == kEarly ? load_l2(" in loads
    for line in re.findall(r"load_l2\(const [^\n]*", text):
        assert "__ldcg(p)" in line
    assert "early ? load_row<T, WIDE, kEarly>" in early
    # only the second product reads early, and it is launched right after the first one, which waits
    assert "if (!GATED) load_weights(first, true)" in early
    tc = body(source("k_mlp_tc.cu"), "launch_mlp_tc_forward")
    assert tc.index("projections(") < tc.index("launch_mlp_few_down(")


def test_bias_sums_come_from_l2_and_end_last():
    text = source("k_mlp_sums.cu")
    kernel = body(text, "column_sums")
    assert kernel.startswith("{") and "if (!q.early) ptx::pdl_wait();" in kernel
    assert kernel.rstrip("} \n").endswith("if (q.early) ptx::pdl_wait();")
    assert "return" not in kernel  # no thread leaves before that wait
    reads = body(text, "load_l2")
    assert reads.count("__ldcg(") == 2
    assert not re.search(r"load_f<", kernel)
    assert "__shared__" not in kernel
    # `early` only after a product that has waited for dg, du and dy
    back = body(source("k_mlp_tc.cu"), "launch_mlp_tc_backward")
    assert "early = n > 0" in back and "if (!e && n > 0) {" in back
    tc = body(source("k_mlp_tc.cu"), "mlp_tc")
    assert tc.index("ptx::pdl_wait();") < tc.index("ptx::pdl_trigger();")
    assert "launch_column_sums(d.dtype, false, false," in source("k_mlp_mma.cu")
