"""Sizes of norm_residual that 32 bits do not hold are refused by the binding, not
passed on in their low bits (no GPU; tensors without memory)."""
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe


def test_more_rows_than_32_bits_count():
    y = torch.empty((2 ** 32 + 3, 8), dtype=torch.bfloat16, device="meta")
    k = torch.empty(2 ** 32 + 3, device="meta")
    for f in (lambda: moe.norm_residual(y, y),
              lambda: moe.norm_residual_backward(y, y, y, dict(r=y, rstd_post=k, rstd_next=k))):
        with pytest.raises(moe.MoeError) as e:
            f()
        assert e.value.status == 2


@pytest.mark.parametrize("T,H,S", [(2 ** 32 + 1, 8, 1), (1, 2 ** 32 + 8, 1), (1, 8, 2 ** 32 + 1), (2 ** 31, 8, 1),
                                   (2 ** 30 + 1, 8, 1), (1, 8, 65537)])
def test_workspace_of_sizes_out_of_range(T, H, S):
    with pytest.raises(moe.MoeError) as e:
        moe.norm_residual_backward_workspace_size(T, H, S)
    assert e.value.status == 2
