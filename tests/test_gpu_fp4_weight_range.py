"""bf16 rows under 4-bit NV weights whose scale exponent lies far from zero, with
rows at both ends of bf16: what stands between the sum of digits and the result
must not leave fp32's range where the result is inside it.

Tolerance of a sum of K terms as in test_gpu_fp4_weight.py: 2 K 2^-24 sum|terms|
for the fp32 accumulation and 2^-35 of a row's largest times sum|w| for its digits;
2^-149, a step of fp32's subnormals, where the result is that small.
"""
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from .test_gpu_fp4_weight import DEV, F64, rows_of, sums, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sigma,exp", [(1e36, -60), (1e36, -20), (2e35, -12), (1e-37, 60), (1e-37, 20),
                                       (1e-37, 4), (1e-37, -60), (1e18, -60), (1e-18, 60)])
def test_scale_exponents_at_the_ends_of_bf16(sigma, exp):
    x, off = rows_of([3, 12], 512, 21, sigma=sigma)
    assert torch.isfinite(x).all() and (x != 0).float().mean() > 0.99
    m, w = weights(2, 256, 512, "nv", 22, exp)
    y = moe.fp4_weight_matmul(x, off, m, out_f32=True)
    assert torch.isfinite(y).all()
    o = off.tolist()
    for g in range(2):
        s, e = sums(x[o[g]:o[g + 1]], w[g])
        assert float(s.abs().max()) < 3e38
        tol = e - 1e-38 + 2.0 ** -149
        assert ((y[o[g]:o[g + 1]].to(F64) - s).abs() <= tol).all()


def test_one_product_at_the_largest_scale():
    """2e35 against 448 * 6 * 2^-12: 1.3e35."""
    K, N = 128, 128
    m = moe.Fp4Matrix(torch.full((1, N, K // 2), 0x77, dtype=torch.uint8, device=DEV),
                      torch.full((moe.fp4_scales_size(N, K, "nv"),), 0x7E, dtype=torch.uint8, device=DEV),
                      "nv", -12)
    x = torch.zeros((1, K), dtype=torch.bfloat16, device=DEV)
    x[0, 5] = 2e35
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    want = float(x[0, 5].to(F64)) * 448 * 6 * 2.0 ** -12
    got = moe.fp4_weight_matmul(x, off, m, out_f32=True).to(F64)
    assert ((got - want).abs() <= 2.0 ** -24 * want).all()
    # an infinity beside it decides the sign: the finite part stays finite
    x[0, 9] = -float("inf")
    assert (moe.fp4_weight_matmul(x, off, m, out_f32=True) == -float("inf")).all()
