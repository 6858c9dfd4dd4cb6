"""A block of the tcgen05 attention kernels that gives up a wait must not end while its own loads
are in flight into its shared memory: each barrier that a load completes on is waited for (with a
limit) on that way out. Read from the source, since such a wait never runs out in a test."""
import re

import pytest

from test_ops_early_start import body, source

KERNELS = [("k_attn_tc_fwd.cu", "attn_tc_forward"), ("k_attn_tc_bwd.cu", "attn_tc_dq"),
           ("k_attn_tc_bwd.cu", "attn_tc_dkv")]


@pytest.mark.parametrize("file,kernel", KERNELS)
def test_every_armed_barrier_is_drained(file, kernel):
    text = body(source(file), kernel)
    load = text[text.index("if (warp == kLoadWarp) {"):text.index("else if (warp == kMmaWarp) {")]
    work, way_out = load.split("if (*abort_flag) {")
    armed = set()
    for name in re.findall(r"mbar_arrive_expect_tx\((\w+),", work):
        for expr in re.findall(rf"const uint32_t {name} = ([^;]+);", work):
            # a barrier may be chosen from others by name
            for inner in re.findall(r"\b(full|bar)\b(?!\[)(?=[;:) ]|$)", expr):
                for e in re.findall(rf"const uint32_t {inner} = ([^;]+);", work):
                    expr += " " + e
            armed |= set(re.findall(r"ctl\.(\w+)", expr))
    assert armed
    drained = set(re.findall(r"drain_bar\(ptx::smem_addr\(&ctl\.(\w+)", way_out))
    at_once = "drain_bar(bar, tails & 1)" in work  # the ragged tiles' own barrier, where it fails
    assert armed - drained - ({"tail"} if at_once else set()) == set(), (armed, drained)
