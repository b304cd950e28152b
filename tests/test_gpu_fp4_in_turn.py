"""4-bit products of a shared expert's many rows (CTA pairs) and of few rows an
expert (single CTAs) behind one another in a stream, as a block issues them: each
starts while the last one ends, and each gives what it gives alone."""
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_pairs_and_single_ctas_in_turn(fmt):
    K, N, E = 512, 384, 16
    g = torch.Generator().manual_seed(41)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)   # noqa: E731
    many, few = rnd(700, K), rnd(50, K)
    one = torch.tensor([0, 700], dtype=torch.int32, device=DEV)
    spread = torch.cat((torch.arange(E, dtype=torch.int32) * 3, torch.tensor([50], dtype=torch.int32))).to(DEV)
    w1, w2 = (moe.fp4_quantize(rnd(n, N, K), fmt) for n in (1, E))
    x1 = moe.fp4_quantize(many, fmt, offsets=one)
    x2 = moe.fp4_quantize(few, fmt, offsets=spread)
    calls = [lambda: moe.fp4_grouped_matmul(x1, one, w1), lambda: moe.fp4_grouped_matmul(x2, spread, w2)]
    alone = []
    for c in calls:
        alone.append(c())
        torch.cuda.synchronize()
    turns = [calls[i & 1]() for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, alone[i & 1]) for i, t in enumerate(turns))
