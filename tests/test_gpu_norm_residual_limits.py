"""norm_residual's backward pass where its inputs hold what a result must not see.

Without a norm after the block d_y = scale d_r gate holds no y: three fp32 factors,
2 roundings of 2^-24 (and one of the product gate * 1), then the type's own.
"""
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from .test_gpu_norm_residual import B, BF, DEV, F32, F64, U, gate_of, make

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("T,H", [(1, 8), (40, 512), (33, 4096), (9, 8192)])
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_gradient_of_an_unnormed_block_holds_none_of_its_output(T, H, xt, yt):
    seq = [0, T // 2, T]
    d = make(T, H, seq, T + H, xt, yt)
    d["y"].view(-1)[1::7] = INF
    d["y"].view(-1)[2::7] = NAN
    d["y"].view(-1)[3::7] = -INF
    kw = dict(gate=d["gate"], scale=0.5, post_norm=False, seq_offsets=d["seq"])
    f = moe.norm_residual(d["x"], d["y"], next_norm=False, **kw)
    g = moe.norm_residual_backward(d["d_r"], None, d["y"], f, **kw)
    assert torch.equal(g["d_x"], d["d_r"])
    want = 0.5 * d["d_r"].to(F64) * gate_of(d, seq, T)
    assert torch.isfinite(g["d_y"]).all()
    tol = (3 * U + (B if yt == BF else U)) * want.abs() + 1e-37
    assert ((g["d_y"].to(F64) - want).abs() <= tol).all()
