"""The router's training operators on logits far from zero, against float64.

Tolerances as in test_gpu_router_grad.py, with one term more.  e = exp(d) of a
difference d = z - m is off by what d log2(e) is rounded by: one rounding of
the difference, one of the product and the constant's own error, 2.3 |d| 2^-24
relative in all.  A gradient's term holds such an e twice (its own and the one
in sum p c), so 5 |d| 2^-24 of its scale, with |d| <= 88: beyond, e is below
fp32's normal range and may be zero (1e-35 absolute covers that with the
factors it meets here).
"""
import numpy as np
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from tests.test_gpu_router_grad import DEV, U, cu, ref_balance, ref_grad

pytestmark = pytest.mark.gpu

# whole vectors on 8, 16 and 32 lanes a token, and rows off the vector size
SHAPES = [(8, 2), (64, 8), (160, 6), (250, 4), (400, 3), (1000, 32)]
ABS = 1e-35


def offset_rows(T, E, offset, seed):
    """Rows shifted by `offset`, rows of equal logits there, and ordinary rows
    between them (in the same warps)."""
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)) * 1.5
    lg = z.astype(np.float32)
    for t in range(T):
        if t % 5 == 1:
            lg[t] = offset
        elif t % 3 != 0:
            lg[t] = (z[t] + offset).astype(np.float32)
    return rng, lg


def farthest(lg):
    d = lg.max(axis=1, keepdims=True).astype(np.float64) - lg
    return d[d <= 88].max()


def top(lg, k):
    return np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)


@pytest.mark.parametrize("E,k", SHAPES)
@pytest.mark.parametrize("offset", [0.0, 100.0, -100.0, 1e3, -1e4, 65504.0, 1e5, -1e6])
def test_weights_of_the_whole_softmax_at_an_offset(E, k, offset):
    """Without renormalisation a slot's weight is its logit's probability among
    all: the two are formed apart and must carry the same factors."""
    T = 41
    rng, lg = offset_rows(T, E, offset, E)
    idx = top(lg, k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    d = moe.gate_topk_backward(cu(lg), cu(idx), cu(dw), renorm=False).cpu().numpy()
    keep = np.ones(T, bool)
    ex, sc = ref_grad(lg.astype(np.float64), idx, dw.astype(np.float64), False, keep, 0.0, [0, T],
                      None, None, 0.0)
    tol = (E + 64 + 5 * farthest(lg)) * U * sc + ABS
    assert (np.abs(d - ex) <= tol).all(), np.max(np.abs(d - ex) / tol)


@pytest.mark.parametrize("E,k", SHAPES)
@pytest.mark.parametrize("offset", [1e3, -1e4, 65504.0, -65504.0, 1e9, -1e9, 3e9, -3e9, 1e10, -1e10,
                                    1e12, -1e12, 1e30, -1e30, 1e37, -1e37, 3e38, -3e38])
def test_any_finite_row(E, k, offset):
    T = 41
    rng, lg = offset_rows(T, E, offset, E + 1)
    idx = top(lg, k)
    seq = np.array([0, 14, 14, T], np.int32)
    keep = rng.random(T) >= 0.1
    dw = rng.standard_normal((T, k)).astype(np.float32) * 1e-2
    lg64 = lg.astype(np.float64)
    args = dict(token_mask=cu(keep), seq_offsets=cu(seq))
    far = farthest(lg)
    b = moe.balance_loss(cu(lg), cu(idx), 0.3, **args)
    loss, c, P, n = ref_balance(lg64, idx, 0.3, keep, seq)
    assert np.array_equal(b["counts"].cpu().numpy(), c)
    err = np.abs(b["prob_mean"].cpu().numpy() - P)
    assert (err <= (1100 + E / 4 + 5 * far) * U * P + ABS).all()
    assert abs(float(b["loss"]) - loss) <= (2200 + E + 10 * far) * U * loss + ABS
    for renorm in (True, False):
        for weights, balance in ((dw, b), (dw, None), (None, b)):
            d = moe.gate_topk_backward(cu(lg), cu(idx), None if weights is None else cu(weights),
                                       renorm=renorm, balance=balance, **args).cpu().numpy()
            ex, sc = ref_grad(lg64, idx, None if weights is None else weights.astype(np.float64),
                              renorm, keep, 0.3, seq, None if balance is None else c, n, 1.0)
            assert (np.abs(d - ex) <= (E + 64 + 5 * far) * U * sc + ABS).all(), (renorm, balance is None)


def test_one_far_row_among_many():
    """A row filled with a mask value far below the others, one of a long
    sequence: its probabilities are uniform, and the sequence's means, loss and
    gradients are those of all its rows."""
    T, E, k = 3000, 64, 8
    rng = np.random.default_rng(3)
    lg = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    lg[1234] = -1e30
    lg[77, 5:] = -1e30                       # experts switched off one by one
    lg[2500] = -1e10
    idx = top(lg, k)
    keep, seq = np.ones(T, bool), [0, T]
    b = moe.balance_loss(cu(lg), cu(idx), 1.0)
    loss, c, P, n = ref_balance(lg.astype(np.float64), idx, 1.0, keep, seq)
    assert (np.abs(b["prob_mean"].cpu().numpy() - P) <= (1100 + E / 4 + 60) * U * P).all()
    assert abs(float(b["loss"]) - loss) <= (2200 + E) * U * loss
    d = moe.gate_topk_backward(cu(lg), cu(idx), balance=b).cpu().numpy()
    ex, sc = ref_grad(lg.astype(np.float64), idx, None, True, keep, 1.0, seq, c, n, 1.0)
    assert (np.abs(d - ex) <= (E + 64 + 5 * farthest(lg)) * U * sc + ABS).all()
