"""How kernels on CTA pairs leave, read from their sources (no GPU): what the
compiler does not check and no run shows reliably."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_expert_routing_fp32_gb300", "csrc")
CALL = "tmem_dealloc_pair("


def calls():
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(re.escape(CALL), src):
            end = src.index("\n}", m.start())            # of the kernel
            out.append((os.path.basename(path), src[max(0, m.start() - 400):m.start()], src[m.start():end]))
    return out


def test_every_pair_kernel_is_found():
    files = [c[0] for c in calls()]
    assert files.count("gemm.cu") == 2 and files.count("fp4_gemm.cu") == 1 and files.count("mlp_train.cu") == 2


@pytest.mark.parametrize("i", range(len(calls())))
def test_pairs_leave_together(i):
    """A pair's tensor memory is given back by both CTAs; until both have done so
    neither leaves its multiprocessor to a CTA that may allocate some of its own."""
    name, before, after = calls()[i]
    assert "cluster_sync_all();" in before, name         # nobody signals or reads the peer any more
    assert "cluster_sync_all();" in after, name
