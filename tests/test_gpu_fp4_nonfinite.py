"""Infinities and NaN in the 4-bit formats.

A block scale's NaN byte (255 with "mx", 127 with "nv") makes the whole block
NaN, dequantised and as an operand of the products alike; a block that holds
an infinity or a NaN is quantised to that byte.
"""
import numpy as np
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from tests import _fp4_ref as ref
from tests.test_gpu_fp4 import DEV, _cuda, _f64, _matrix, _rows, _sums

pytestmark = pytest.mark.gpu
NAN_BYTE = {"mx": 255, "nv": 127}


def _poison(m, fmt, n, K, offsets, places):
    """Scale bytes of (row, block) made NaN in place."""
    pos = ref.scale_positions(n, K // ref.BLOCK[fmt], offsets)
    for r, b in places:
        m.sf[int(pos[r, b])] = NAN_BYTE[fmt]


def _spread(places, n, K, fmt):
    bad = np.zeros((n, K), bool)
    for r, b in places:
        bad[r, b * ref.BLOCK[fmt]:(b + 1) * ref.BLOCK[fmt]] = True
    return bad


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("offsets", [None, [0, 40, 40, 200]])
def test_nan_scales_dequantise_to_nan(fmt, offsets):
    n, K = 200, 1152
    x = _rows(n, K, 3)
    x[7] = 0.0                                          # codes of zero under a NaN scale
    off = None if offsets is None else np.array(offsets, np.int32)
    m, val = _matrix(_f64(x), fmt, 0, off)
    places = [(0, 0), (7, 1), (39, K // ref.BLOCK[fmt] - 1), (130, 5), (131, 5), (199, 2)]
    _poison(m, fmt, n, K, off, places)
    got = _f64(moe.fp4_dequantize(m, None if off is None else _cuda(off)))
    bad = _spread(places, n, K, fmt)
    assert np.isnan(got[bad]).all()
    assert np.array_equal(got[~bad], _f64(ref.bf16(val))[~bad])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sizes", [[40, 3], [700, 5]])          # one CTA, CTA pairs
def test_nan_scales_make_rows_and_columns_nan(fmt, sizes):
    K, N = 384, 256
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n, G = int(off[-1]), len(sizes)
    x = _rows(n, K, 5)
    x[2] = 0.0
    a, av = _matrix(_f64(x), fmt, 0, off)
    w, wv = _matrix(_f64(_rows(G * N, K, 6, 0.5)), fmt, 0)
    w.q, wv = w.q.view(G, N, K // 2), wv.reshape(G, N, K)
    rows, cols = [(2, 1), (n - 1, 0), (17, K // ref.BLOCK[fmt] - 1)], [(3, 0), (N + 200, 2)]
    _poison(a, fmt, n, K, off, rows)
    _poison(w, fmt, G * N, K, None, cols)
    y, s = _sums(off, av, wv, n)
    bad = np.zeros((n, N), bool)
    bad[[r for r, _ in rows]] = True
    for c, _ in cols:
        g = c // N
        bad[off[g]:off[g + 1], c % N] = True
    got = _f64(moe.fp4_grouped_matmul(a, _cuda(off), w, out_f32=True))
    assert np.isnan(got[bad]).all()
    assert (np.abs(got - y)[~bad] <= ((K + 8) * 2.0 ** -23 * s)[~bad]).all()


@pytest.mark.parametrize("fmt,exp", [("mx", 0), ("nv", 0), ("nv", -9), ("nv", 60)])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("k", [1, 3])
def test_quantised_infinities_and_nan_stay_visible(fmt, exp, value, k):
    T, K = 70, 640
    x = _rows(T, K, 7, 2.0 ** min(exp, 30))
    B = ref.BLOCK[fmt]
    places = [(0, 0), (33, 3), (69, K // B - 1)]
    clean = _f64(x)
    for i, (r, b) in enumerate(places):
        x[r, b * B + (5 * i) % B] = value
        clean[r, b * B:(b + 1) * B] = 0.0
    rng = np.random.default_rng(8)
    rows = rng.permutation(T * k).astype(np.int32)
    off = np.array([0, 50, T * k], np.int32)
    m = moe.fp4_quantize(x.to(DEV), fmt, exp, row_idx=_cuda(rows), k=k, offsets=_cuda(off))
    got = _f64(moe.fp4_dequantize(m, _cuda(off)))[rows].reshape(T, k, K)
    val = _f64(ref.bf16(ref.quantize(clean, fmt, exp)[2]))
    bad = _spread(places, T, K, fmt)
    for j in range(k):
        assert np.isnan(got[:, j][bad]).all()
        assert np.array_equal(got[:, j][~bad], val[~bad])
    pos = ref.scale_positions(T * k, K // B, off)
    sf = m.sf.cpu().numpy()
    assert all(sf[pos[rows[r * k + j], b]] == NAN_BYTE[fmt] for r, b in places for j in range(k))


@pytest.mark.parametrize("fmt,e", [("mx", 0), ("nv", 30)])
@pytest.mark.parametrize("sizes", [[0, 40, 129, 3], [700, 5]])  # one CTA, CTA pairs
def test_overflowing_act_stays_visible_in_4_bits(fmt, e, sizes):
    """Gate and up sums near 2^64: some act values pass bf16's range.  The 4-bit
    form has NaN blocks exactly where the bf16 form is not finite, the other
    blocks as they are, and the second product NaN rows exactly there."""
    K = H = I = 256
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n, G = int(off[-1]), len(sizes)
    x = _f64(_rows(n, K, 9)) * 2.0 ** 29
    x[::3] *= 2.0 ** -20                               # rows that stay finite
    a, _ = _matrix(_f64(ref.bf16(x)), fmt, e, off)
    w, _ = _matrix(_f64(ref.bf16(_f64(_rows(G * 2 * I, K, 10)) * 2.0 ** 29)), fmt, e)
    w.q = w.q.view(G, 2 * I, K // 2)
    w2, _ = _matrix(_f64(_rows(G * H, I, 11, 2.0 ** -20)), fmt, -20 if fmt == "nv" else 0)
    w2.q = w2.q.view(G, H, I // 2)
    offc, act_exp = _cuda(off), 60 if fmt == "nv" else 0
    act = _f64(moe.fp4_grouped_swiglu(a, offc, w))
    q = moe.fp4_grouped_swiglu(a, offc, w, quantize=True, scale_exp=act_exp)
    B = ref.BLOCK[fmt]
    bad = ~np.isfinite(act.reshape(n, I // B, B)).all(axis=2)
    assert bad.any() and not bad.all(axis=1).all()
    clean = np.where(np.repeat(bad, B, axis=1), 0.0, act)
    code, byte, val = ref.quantize(clean, fmt, act_exp)
    sf = q.sf.cpu().numpy()[ref.scale_positions(n, I // B, off)]
    assert (sf[bad] == NAN_BYTE[fmt]).all() and np.array_equal(sf[~bad], byte[~bad])
    codes = q.q.cpu().numpy().reshape(n, I // B, B // 2)
    assert np.array_equal(codes[~bad], ref.pack(code).reshape(n, I // B, B // 2)[~bad])
    act4, y = moe.fp4_grouped_mlp(a, offc, w, w2, y_f32=True, act_exp=act_exp)
    assert torch.equal(act4.q, q.q)
    lost = bad.any(axis=1)
    got = _f64(y)
    assert np.isnan(got[lost]).all() and np.isfinite(got[~lost]).all()
