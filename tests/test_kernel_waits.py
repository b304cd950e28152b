"""What follows a wait that gives up, read from the kernels' sources (no GPU; a wait
that runs out in one warp and not in the next cannot be staged).

A role of several warps whose loop holds barriers for all of them must leave it with
all of them: were one to go alone, the others would wait at a barrier it never
reaches, and the bounded wait would end in an endless kernel.  A warp likewise: its
lanes poll one by one, and what follows (tensor memory loads above all) takes all 32."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_expert_routing_fp32_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_epilogue_with_barriers_leaves_its_loop_as_one():
    src = source("fp4_weight.cu")
    role = src[src.index("} else if (warp >= 4) {"):src.index("tmem_dealloc(")]
    assert "bar.sync 1, 128" in role
    waits = re.findall(r"(\w+)\(\s*wait_phase\(", role)
    assert len(waits) == len(re.findall(r"wait_phase\(", role)) == 1
    assert waits == ["all_warps"]
    body = src[src.index("bool all_warps("):]
    assert "bar.red.and.pred" in body[:body.index("\n}")]


# barriers that whole warps wait on: accumulators (tfull), h, rows to be zeroed
@pytest.mark.parametrize("name,waits", [("gemm.cu", 3), ("fp4_gemm.cu", 1), ("mlp_train.cu", 5)])
def test_warps_agree_on_a_wait(name, waits):
    src = source(name)
    found = re.findall(r"(\w+)\(\s*(?:wait_phase|wait_acc|mbar_wait_bounded)\(\s*&?(?:tfull|h_full|tail)\b", src)
    assert found == ["whole_warp"] * waits
