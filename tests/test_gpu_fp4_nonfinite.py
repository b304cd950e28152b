"""NaN in the 4-bit formats.

A block scale's NaN byte (255 with "mx", 127 with "nv") makes the whole block
NaN, dequantised and as an operand of the products alike.
"""
import numpy as np
import pytest

import moe_expert_routing_fp32_gb300 as moe
from tests import _fp4_ref as ref
from tests.test_gpu_fp4 import _cuda, _f64, _matrix, _rows, _sums

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
