"""4-bit operands on the GPU against the 64-bit reference in _fp4_ref.py.

Quantisation and dequantisation are exact (codes, scale bytes and values bit
for bit).  A product's fp32 sum of K exact terms is allowed one fp32 step per
addition, (K + 8) 2^-23 sum |a w|, and the output's own rounding, half a step:
2^-8 (bf16) of the value.  SiLU(g) u from sums off by dg, du: |SiLU'| <= 1.1,
so 1.1 |u| dg + |SiLU(g)| du, 2^-19 of the value for the exponential and the
division, and the output's half step.
"""
import numpy as np
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from tests import _fp4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _rows(n, K, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, K)) * scale
    x[:, ::37] *= 11.0
    return ref.bf16(x)


def _cuda(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dt is None else t.to(dt)).to(DEV)


def _f64(t):
    return t.double().cpu().numpy()


def _matrix(x, fmt, exp, offsets=None):
    """Reference-quantised operand on the GPU and its float64 values.  Bytes
    of the layout that belong to no row hold 0xFF (a NaN scale)."""
    code, byte, val = ref.quantize(x, fmt, exp)
    G = 0 if offsets is None else len(offsets) - 1
    sf = ref.place(byte, offsets, moe.fp4_scales_size(len(x), x.shape[1], fmt, G), fill=0xFF)
    return moe.Fp4Matrix(_cuda(ref.pack(code)), _cuda(sf), fmt, exp), val


# ---------------------------------------------------------------- conversions
def _edge_rows(K):
    """Rows of ties, saturating and vanishing blocks, signed zeros, single
    values, powers of two and their neighbours, subnormals, the largest."""
    rng = np.random.default_rng(7)
    rows = [np.zeros(K), -np.zeros(K)]
    for s in (1.0, 2.0 ** -20, 2.0 ** 30, 3.0, 448.0 * 6, 2.0 ** -11, 2.0 ** 120, 2.0 ** -126):
        grid = np.array([0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5])
        r = np.zeros(K)
        r[:] = rng.choice(np.concatenate([grid, -grid]), K) * s
        rows.append(r)
        one = np.zeros(K)
        one[K // 2] = s
        rows.append(one)
        rows.append(np.full(K, s))
        rows.append(np.full(K, -s * (1 - 2.0 ** -8)))
    rows.append(np.full(K, 2.0 ** -133))
    rows.append(rng.standard_normal(K) * 2.0 ** -130)
    rows.append(np.full(K, 3.3895313892515355e38))
    return ref.bf16(np.array(rows))


@pytest.mark.parametrize("fmt,exp", [("mx", 0), ("nv", 0), ("nv", -7), ("nv", 60), ("nv", -60)])
@pytest.mark.parametrize("K", [128, 256, 1152, 4096])
def test_quantize_is_exact(fmt, exp, K):
    x = torch.cat([_edge_rows(K), _rows(150, K, 1), _rows(33, K, 2, 0.02)])
    m = moe.fp4_quantize(x.to(DEV), fmt, exp)
    v = moe.fp4_dequantize(m)
    code, byte, val = ref.quantize(_f64(x), fmt, exp)
    assert np.array_equal(m.q.cpu().numpy(), ref.pack(code))
    pos = ref.scale_positions(len(x), byte.shape[1])
    assert np.array_equal(m.sf.cpu().numpy()[pos], byte)
    assert torch.equal(v.cpu(), ref.bf16(val))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("n", [0, 1, 31, 128, 129, 1000])
def test_quantize_row_counts(fmt, n):
    x = _rows(n, 256, 3)
    m = moe.fp4_quantize(x.to(DEV), fmt)
    v = moe.fp4_dequantize(m)
    assert m.q.shape == (n, 128) and v.shape == (n, 256)
    assert torch.equal(v.cpu(), ref.bf16(ref.quantize(_f64(x), fmt)[2]))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,K,E,k", [(1, 128, 4, 1), (77, 384, 13, 3), (500, 1280, 1000, 2),
                                     (300, 128, 64, 32), (64, 2176, 8, 8)])
def test_quantize_into_expert_order(fmt, T, K, E, k):
    x = _rows(T, K, 4)
    rng = np.random.default_rng(5)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    if E > 20:
        idx = np.sort(idx, axis=1)
    r = moe.init_routing(_cuda(idx), x.to(DEV), E)
    m = moe.fp4_quantize(x.to(DEV), fmt, row_idx=r["row_idx"], k=k, offsets=r["offsets"])
    direct = ref.quantize(_f64(r["expanded_x"]), fmt)
    assert np.array_equal(m.q.cpu().numpy(), ref.pack(direct[0]))
    pos = ref.scale_positions(T * k, K // ref.BLOCK[fmt], r["offsets"].cpu().numpy())
    assert np.array_equal(m.sf.cpu().numpy()[pos], direct[1])
    v = moe.fp4_dequantize(m, r["offsets"])
    assert torch.equal(v.cpu(), ref.bf16(direct[2]))


def test_rows_without_a_place_are_left_alone():
    """Negative rows, rows behind the last group and rows past the end."""
    T, K, k = 6, 128, 2
    x = _rows(T, K, 6).to(DEV)
    rows = torch.tensor([0, 1, -1, 3, 4, 5, 6, 7, 8, 9, 99, 11], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    st = moe.new_status(DEV)
    size = moe.fp4_scales_size(T * k, K, "nv", 2)
    q = torch.full((T * k, K // 2), 0xA5, dtype=torch.uint8, device=DEV)
    sf = torch.full((size,), 0xA5, dtype=torch.uint8, device=DEV)
    m = moe.Fp4Matrix(q, sf, "nv")
    moe._call("moe_fp4_quantize", moe._ptr(x), T, K, moe._ptr(rows), k, moe._ptr(off), 2,
              moe._fp4_arg(m, "out", 2, x.device), moe._ptr(st), moe._stream(x.device))
    assert int(st.item()) == moe.DEV_BAD_OFFSETS
    for r in (2, 8, 9, 10, 11):
        assert (q[r] == 0xA5).all(), r
    code = ref.pack(ref.quantize(_f64(x), "nv")[0])
    for r in (0, 1, 3, 4, 5, 6, 7):
        t = rows.tolist().index(r) // k
        assert np.array_equal(q[r].cpu().numpy(), code[t]), r
    pos = ref.scale_positions(T * k, 8, [0, 4, 8])
    touched = set(pos[[0, 1, 3, 4, 5, 6, 7]].reshape(-1).tolist())
    s = sf.cpu().numpy()
    assert all(s[i] == 0xA5 for i in range(size) if i not in touched)
    out = torch.full((T * k, K), 7.0, dtype=torch.bfloat16, device=DEV)
    moe._call("moe_fp4_dequantize", moe._fp4_arg(m, "m", 2, x.device), T * k, K, moe._ptr(off), 2,
              moe._ptr(out), moe._stream(x.device))
    assert (out[8:] == 7.0).all()


# ------------------------------------------------------------------- products
GROUPS = {
    "one": [1],
    "ragged": [0, 1, 127, 128, 129, 0, 300, 3],
    "single-tokens": [1] * 9 + [0] * 4 + [2],
    "none": [0, 0, 0],
    "big": [700, 5],
}


def _problem(sizes, K, N, fmt, ea, ew, seed, start=0, extra=0, wscale=0.02):
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + start
    n = int(off[-1]) + extra
    G = len(sizes)
    a, av = _matrix(_f64(_rows(n, K, seed)), fmt, ea, off)
    w, wv = _matrix(_f64(_rows(G * N, K, seed + 1, wscale)), fmt, ew)
    w.q = w.q.view(G, N, K // 2)
    return off, n, a, av, w, wv.reshape(G, N, K)


def _sums(off, av, wv, n):
    """Exact products and their bound's sum |a w| in float64."""
    N = wv.shape[1]
    y, s = np.zeros((n, N)), np.zeros((n, N))
    for g in range(len(off) - 1):
        r = slice(off[g], off[g + 1])
        y[r] = av[r] @ wv[g].T
        s[r] = np.abs(av[r]) @ np.abs(wv[g]).T
    return y, s


SHAPES = [("ragged", 128, 128), ("one", 128, 128), ("ragged", 384, 256), ("one", 256, 384), ("single-tokens", 1152, 128),
          ("none", 128, 128), ("big", 640, 512), ("ragged", 2048, 640)]


@pytest.mark.parametrize("fmt,ea,ew", [("mx", 0, 0), ("nv", 0, -6)])
@pytest.mark.parametrize("groups,K,N", SHAPES)
@pytest.mark.parametrize("f32", [False, True])
def test_grouped_matmul(fmt, ea, ew, groups, K, N, f32):
    off, n, a, av, w, wv = _problem(GROUPS[groups], K, N, fmt, ea, ew, 11, extra=3)
    st = moe.new_status(DEV)
    dt = torch.float32 if f32 else torch.bfloat16
    out = torch.full((n, N), -77.0, dtype=dt, device=DEV)
    moe.fp4_grouped_matmul(a, _cuda(off), w, out_f32=f32, out=out, status=st)
    assert int(st.item()) == 0
    y, s = _sums(off, av, wv, n)
    got = _f64(out)
    end = off[-1]
    assert (got[end:] == -77.0).all()                  # rows behind the last group
    tol = (K + 8) * 2.0 ** -23 * s[:end] + (0.0 if f32 else 2.0 ** -8) * np.abs(y[:end])
    assert (np.abs(got[:end] - y[:end]) <= tol).all()


def _check_act(got, g, u, sg, su, K):
    sig = 1.0 / (1.0 + np.exp(-g))
    act = g * sig * u
    d = (K + 8) * 2.0 ** -23
    tol = 1.1 * np.abs(u) * d * sg + np.abs(g * sig) * d * su + (2.0 ** -19 + 2.0 ** -8) * np.abs(act)
    # second order of the two errors, and bf16's smallest steps
    tol = tol + 1.1 * d * d * sg * su + 2.0 ** -134
    assert (np.abs(got - act) <= tol).all(), np.max(np.abs(got - act) - tol)


@pytest.mark.parametrize("fmt,ea,ew", [("mx", 0, 0), ("nv", 3, -9)])
@pytest.mark.parametrize("groups,K,I", SHAPES)
def test_grouped_swiglu_and_its_quantised_form(fmt, ea, ew, groups, K, I):
    off, n, a, av, w, wv = _problem(GROUPS[groups], K, 2 * I, fmt, ea, ew, 21, extra=2)
    st = moe.new_status(DEV)
    offc = _cuda(off)
    out = torch.full((n, I), -77.0, dtype=torch.bfloat16, device=DEV)
    moe.fp4_grouped_swiglu(a, offc, w, out=out, status=st)
    y, s = _sums(off, av, wv, n)
    end = off[-1]
    got = _f64(out)
    assert (got[end:] == -77.0).all()
    _check_act(got[:end], y[:end, :I], y[:end, I:], s[:end, :I], s[:end, I:], K)
    # the quantised form holds exactly those bf16 values in 4 bits
    fused = moe.fp4_grouped_swiglu(a, offc, w, quantize=True, scale_exp=0, status=st)
    code, byte, val = ref.quantize(got[:end], fmt)
    assert int(st.item()) == 0
    assert np.array_equal(fused.q.cpu().numpy()[:end], ref.pack(code))
    pos = ref.scale_positions(n, I // ref.BLOCK[fmt], off)[:end]
    assert np.array_equal(fused.sf.cpu().numpy()[pos], byte)
    # and mlp is the two products in a row
    H = K
    w2, w2v = _matrix(_f64(_rows((len(off) - 1) * H, I, 31, 0.05)), fmt, 0 if fmt == "mx" else ew)
    w2.q = w2.q.view(len(off) - 1, H, I // 2)
    act, ym = moe.fp4_grouped_mlp(a, offc, w, w2, y_f32=True, status=st)
    y2 = moe.fp4_grouped_matmul(fused, offc, w2, out_f32=True, status=st)
    assert torch.equal(act.q[:end], fused.q[:end]) and torch.equal(ym[:end], y2[:end])
    ex, sm = _sums(off, val if n == end else np.vstack([val, np.zeros((n - end, I))]),
                   w2v.reshape(len(off) - 1, H, I), n)
    assert (np.abs(_f64(ym)[:end] - ex[:end]) <= (I + 8) * 2.0 ** -23 * sm[:end]).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("start,sizes", [(5, [100, 0, 200]), (130, [1, 128])])
def test_groups_may_start_behind_row_zero(fmt, start, sizes):
    off, n, a, av, w, wv = _problem(sizes, 256, 256, fmt, 0, 0, 41, start=start)
    out = torch.full((n, 256), -77.0, device=DEV)
    moe.fp4_grouped_matmul(a, _cuda(off), w, out_f32=True, out=out)
    y, s = _sums(off, av, wv, n)
    got = _f64(out)
    assert (got[:start] == -77.0).all()
    assert (np.abs(got - y)[start:] <= (264 * 2.0 ** -23 * s)[start:]).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("groups,rows", [(3, 2500), (2, 4000)])
def test_many_rows_per_group(fmt, groups, rows):
    """Large groups (the CTA-pair tiles), ragged ends, against fp32 products
    of the dequantised operands on the GPU (K = 512 terms, each side within
    its own K 2^-23 sum |a w|)."""
    K, N = 512, 768
    sizes = [rows, 1, rows - 129, 257][:groups + 1]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n, G = int(off[-1]), len(sizes)
    x = _rows(n, K, 51).to(DEV)
    wx = _rows(G * N, K, 52, 0.02).to(DEV)
    ident = torch.arange(n, dtype=torch.int32, device=DEV)
    offc = _cuda(off)
    a = moe.fp4_quantize(x, fmt, row_idx=ident, offsets=offc)
    w = moe.fp4_quantize(wx.view(G, N, K), fmt, 0 if fmt == "mx" else -6)
    st = moe.new_status(DEV)
    y = moe.fp4_grouped_matmul(a, offc, w, out_f32=True, status=st).double()
    av = moe.fp4_dequantize(a, offc).double()
    wv = moe.fp4_dequantize(w).double()
    act = moe.fp4_grouped_swiglu(a, offc, w, status=st).double().cpu().numpy()
    q = moe.fp4_grouped_swiglu(a, offc, w, quantize=True, status=st)
    assert int(st.item()) == 0
    for g in range(G):
        r = slice(int(off[g]), int(off[g + 1]))
        ex = av[r] @ wv[g].T
        s = av[r].abs() @ wv[g].abs().T
        assert ((y[r] - ex).abs() <= (K + 8) * 2.0 ** -23 * s).all()
        e, sm = ex.cpu().numpy(), s.cpu().numpy()
        h = N // 2
        _check_act(act[r], e[:, :h], e[:, h:], sm[:, :h], sm[:, h:], K)
    code, byte, _ = ref.quantize(act, fmt)
    assert np.array_equal(q.q.cpu().numpy(), ref.pack(code))
    pos = ref.scale_positions(n, N // 2 // ref.BLOCK[fmt], off)
    assert np.array_equal(q.sf.cpu().numpy()[pos], byte)


def test_offsets_past_32_bits():
    """More than 2^31 bytes of codes and 2^32 of rows in and values out: the
    rows of a repeated block give that block's bytes everywhere."""
    K, block = 4096, 4096
    n = 2 ** 20 + block + 257
    G = 2
    x = _rows(block, K, 91).to(DEV)
    big = x.repeat(n // block + 1, 1)[:n].contiguous()
    m = moe.fp4_quantize(big, "nv")
    one = moe.fp4_quantize(x, "nv")
    assert torch.equal(m.q[-257:], one.q[:257]) and torch.equal(m.q[2 ** 20:2 ** 20 + block], one.q)
    v = moe.fp4_dequantize(m)
    assert torch.equal(v[-257:], moe.fp4_dequantize(one)[:257])
    del v
    # the same rows in two groups, the second one far behind
    off = torch.tensor([0, block, n], dtype=torch.int32, device=DEV)
    ident = torch.arange(n, dtype=torch.int32, device=DEV)
    a = moe.fp4_quantize(big, "nv", row_idx=ident, offsets=off)
    del big
    w = moe.fp4_quantize(_rows(128, K, 92, 0.02).to(DEV).repeat(G * 8, 1).view(G, 1024, K), "nv", -6)
    st = moe.new_status(DEV)
    y = moe.fp4_grouped_matmul(a, off, w, out_f32=True, status=st)
    assert int(st.item()) == 0 and y.numel() * 4 > 2 ** 32
    assert torch.equal(y[:block, :128], y[2 ** 20:2 ** 20 + block, 896:])
    assert torch.equal(y[-257:], y[:257])
    ex = moe.fp4_dequantize(one).double() @ moe.fp4_dequantize(w)[0, :128].double().T
    s = moe.fp4_dequantize(one).double().abs() @ moe.fp4_dequantize(w)[0, :128].double().abs().T
    assert ((y[:block, :128].double() - ex).abs() <= (K + 8) * 2.0 ** -23 * s).all()


def test_more_groups_than_a_pair_kernel_lists():
    """1024 groups of more than 128 rows each: the one-CTA tiles take them."""
    G, rows, K, N = 1024, 130, 128, 128
    off = np.arange(G + 1, dtype=np.int32) * rows
    offc = _cuda(off)
    ident = torch.arange(G * rows, dtype=torch.int32, device=DEV)
    a = moe.fp4_quantize(_rows(G * rows, K, 95).to(DEV), "mx", row_idx=ident, offsets=offc)
    w = moe.fp4_quantize(_rows(G * N, K, 96).to(DEV).view(G, N, K), "mx")
    y = moe.fp4_grouped_matmul(a, offc, w, out_f32=True)
    av = moe.fp4_dequantize(a, offc).double().view(G, rows, K)
    wv = moe.fp4_dequantize(w).double()
    ex, s = av @ wv.transpose(1, 2), av.abs() @ wv.abs().transpose(1, 2)
    assert ((y.double().view(G, rows, N) - ex).abs() <= (K + 8) * 2.0 ** -23 * s).all()


@pytest.mark.parametrize("sizes", [[64, 64], [1500, 600]])      # one CTA, CTA pairs
def test_bad_offsets_are_reported_and_nothing_written(sizes):
    off, n, a, av, w, wv = _problem(sizes, 128, 128, "mx", 0, 0, 61)
    x, y = sizes
    for bad in ([0, n + 16, n], [0, x, n + 1000], [-1, x, n], [x, 0, n]):
        st = moe.new_status(DEV)
        out = torch.full((n, 128), 3.0, device=DEV)
        offc = torch.tensor(bad, dtype=torch.int32, device=DEV)
        moe.fp4_grouped_matmul(a, offc, w, out_f32=True, out=out, status=st)
        assert int(st.item()) == moe.DEV_BAD_OFFSETS
        assert (out == 3.0).all()
    st = moe.new_status(DEV)
    moe.fp4_grouped_matmul(a, _cuda(off), w, out_f32=True, out=out, status=st)
    ex, s = _sums(off, av, wv, n)
    assert int(st.item()) == 0
    assert (np.abs(_f64(out) - ex) <= 136 * 2.0 ** -23 * s).all()


def test_streams_graphs_and_repeats_give_the_same_bytes():
    """Two calls at once on two streams, a captured call replayed with new
    contents and next to another graph, and repeats: the same bytes."""
    sizes, K, I = [300, 0, 129, 2000], 512, 256
    off, n, a, av, w, wv = _problem(sizes, K, 2 * I, "nv", 0, -6, 71)
    off2, n2, a2, _, w2, _ = _problem([1500, 40], K, 2 * I, "nv", 0, -6, 81)
    offc, off2c = _cuda(off), _cuda(off2)
    want = moe.fp4_grouped_swiglu(a, offc, w)
    want2 = moe.fp4_grouped_swiglu(a2, off2c, w2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got, got2 = [], []
    for _ in range(4):
        with torch.cuda.stream(s1):
            got.append(moe.fp4_grouped_swiglu(a, offc, w))
        with torch.cuda.stream(s2):
            got2.append(moe.fp4_grouped_swiglu(a2, off2c, w2))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got) and all(torch.equal(t, want2) for t in got2)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = moe.fp4_grouped_swiglu(a, offc, w)
    with torch.cuda.graph(g2):
        o2 = moe.fp4_grouped_swiglu(a2, off2c, w2)
    for _ in range(3):
        o1.zero_()
        o2.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, want) and torch.equal(o2, want2)
    keep = a.q.clone()
    a.q.copy_(torch.flip(keep, [0]))
    fresh = moe.fp4_grouped_swiglu(a, offc, w)
    g1.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, fresh) and not torch.equal(fresh, want)
