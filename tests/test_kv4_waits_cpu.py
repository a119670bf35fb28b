"""Waits with a limit in the tcgen05 attention kernel, from its source: once a wait has run out, the warps of a thread
block may be at different places of a step, so that a barrier without a limit among the steps could wait forever."""
import os
import re

from quantized_verification_gb300 import build


def test_no_barrier_without_limit_among_the_steps():
    with open(os.path.join(build.CSRC, "k_attn_kv4_tc.cu")) as f:
        source = f.read()
    steps = source[source.index("// ---- 128 positions at a time"):source.index("// ---- the rows' sums, and the weights")]
    code = re.sub(r"//[^\n]*", "", steps)
    assert "wait_for(bar_g" in code and "wait_for(bar_o" in code
    for barrier in ("__syncthreads", "named_bar_sync", "bar.sync", "barrier.sync", "mbar_wait(", "cluster_wait"):
        assert barrier not in code, barrier
    # whoever issues products or requests records decides as a whole warp
    for decision in re.findall(r"if \(([^\n]*elect_one\(\)[^\n]*)\) \{", code):
        assert "__all_sync" in decision, decision
