"""The 16-column format's matrix exponents through the products, act's own among
them, and SwiGLU at the ends of the range that its operands' exponents may add
up to.

Sums as in test_gpu_fp4.py, off by at most (K + 8) 2^-23 sum |a w|.  SiLU of a
gate g: the exponential of the rounded g log2(e) is off by 2.3 |g| 2^-24, the
exponential, sum, reciprocal and products by 16 2^-24 together; below
g = -87.3 the reciprocal of 1 + e^-g (above 2^126) may be zero, a loss of at
most |g| 2^-126.  Then bf16's half step.
"""
import numpy as np
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from tests import _fp4_ref as ref
from tests.test_gpu_fp4 import _cuda, _f64, _matrix, _rows, _sums

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def check_act(got, g, u, sg, su, K):
    with np.errstate(over="ignore"):
        silu = g / (1.0 + np.exp(-g))
    d = (K + 8) * 2.0 ** -23
    near = np.where(g < 0, np.minimum(np.abs(g), 110.0), 0.0)
    tol = (1.1 * np.abs(u) * d * sg + np.abs(silu) * d * su + 1.1 * d * d * sg * su +
           ((2.3 * near + 16) * U + 2.0 ** -8) * np.abs(silu * u) + near * np.abs(u) * 2.0 ** -126 +
           2.0 ** -134)
    assert (np.abs(got - silu * u) <= tol).all(), np.max(np.abs(got - silu * u) / tol)


@pytest.mark.parametrize("sizes", [[40, 3], [700, 5]])          # one CTA, CTA pairs
@pytest.mark.parametrize("ea,ew", [(30, 30), (60, 0), (-30, -30), (0, -60), (-60, 60), (3, -9), (4, 4)])
def test_exponents_of_the_products(sizes, ea, ew):
    K = H = I = 256
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n, G = int(off[-1]), len(sizes)
    # values around 2^-4 of the unit: gates of about 2^(ea + ew), act below 2^126
    a, av = _matrix(_f64(_rows(n, K, 1, 2.0 ** (ea - 4))), "nv", ea, off)
    w, wv = _matrix(_f64(_rows(G * 2 * I, K, 2, 2.0 ** (ew - 4))), "nv", ew)
    w.q, wv = w.q.view(G, 2 * I, K // 2), wv.reshape(G, 2 * I, K)
    w2, w2v = _matrix(_f64(_rows(G * H, I, 3, 2.0 ** 3)), "nv", 5)
    w2.q, w2v = w2.q.view(G, H, I // 2), w2v.reshape(G, H, I)
    offc = _cuda(off)
    y, s = _sums(off, av, wv, n)
    got = _f64(moe.fp4_grouped_matmul(a, offc, w, out_f32=True))
    assert (np.abs(got - y) <= (K + 8) * 2.0 ** -23 * s).all()
    act = _f64(moe.fp4_grouped_swiglu(a, offc, w))
    check_act(act, y[:, :I], y[:, I:], s[:, :I], s[:, I:], K)
    held = 0
    for exp in (-60, -7, 0, 5, 60):
        q = moe.fp4_grouped_swiglu(a, offc, w, quantize=True, scale_exp=exp)
        code, byte, val = ref.quantize(act, "nv", exp)
        assert np.array_equal(q.q.cpu().numpy(), ref.pack(code))
        pos = ref.scale_positions(n, I // 16, off)
        assert np.array_equal(q.sf.cpu().numpy()[pos], byte)
        act4, ym = moe.fp4_grouped_mlp(a, offc, w, w2, y_f32=True, act_exp=exp)
        assert act4.scale_exp == exp and torch.equal(act4.q, q.q)
        ex, sm = _sums(off, val, w2v, n)
        # a sum whose terms all lie in fp32's subnormal range is off by its steps
        assert (np.abs(_f64(ym) - ex) <= (I + 8) * 2.0 ** -23 * sm + I * 2.0 ** -149).all()
        held += bool(val.any())
    assert held >= (0 if ea + ew < -30 else 1)


@pytest.mark.parametrize("sizes", [[40, 3], [700, 5]])
def test_gates_where_the_exponential_overflows(sizes):
    """Gates from -200 to 200 against ups of 1 and of 2^100: large ones pass
    through, those below -87.3 vanish."""
    K, I = 128, 128
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n, G = int(off[-1]), len(sizes)
    x = np.zeros((n, K))
    x[:, 0] = np.linspace(-200, 200, n)                # a block of its own: the gate
    x[:, 64] = np.where(np.arange(n) % 2, 1.0, 2.0 ** 100)
    a, av = _matrix(_f64(ref.bf16(x)), "mx", 0, off)
    wx = np.zeros((G, 2 * I, K))
    wx[:, :I, 0] = 1.0
    wx[:, I:, 64] = 1.0
    w, wv = _matrix(wx.reshape(G * 2 * I, K), "mx", 0)
    w.q, wv = w.q.view(G, 2 * I, K // 2), wv.reshape(G, 2 * I, K)
    y, s = _sums(off, av, wv, n)
    got = _f64(moe.fp4_grouped_swiglu(a, _cuda(off), w))
    assert np.isfinite(got).all()
    check_act(got, y[:, :I], y[:, I:], s[:, :I], s[:, I:], K)
