"""bf16 rows times 4-bit weights against float64.

Tolerance of a sum of K terms: 2 K 2^-24 sum|terms| for the fp32 accumulation
(the tensor cores may truncate; the joins of digits and partial sums are within
that), 2^-35 of a row's largest (a block's at most) times sum|w| for the row's
digits, and the result's own rounding (bf16: 2^-8).  SwiGLU propagates both sums' errors with
|SiLU'| <= 1.1 and adds 2^-18 for the hardware exponential and reciprocal at
gates down to -20.
"""
import numpy as np
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from . import _fp4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, B = 2.0 ** -24, 2.0 ** -8
F64 = torch.float64


def weights(G, rows, K, fmt, seed, exp=0, sigma=1.0):
    """A random 4-bit matrix -> (Fp4Matrix, values float64 [G, rows, K])."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (G * rows, K)).astype(np.uint8)
    nb = K // ref.BLOCK[fmt]
    byte = rng.integers(117, 128, (G * rows, nb)) if fmt == "mx" else rng.integers(1, 100,
                                                                                   (G * rows, nb))
    byte = byte.astype(np.uint8)
    sf = ref.place(byte, None, moe.fp4_scales_size(G * rows, K, fmt))
    m = moe.Fp4Matrix(torch.from_numpy(ref.pack(code)).view(G, rows, K // 2).to(DEV),
                      torch.from_numpy(sf).to(DEV), fmt, exp)
    return m, torch.from_numpy(ref.values(code, byte, fmt, exp)).view(G, rows, K).to(DEV)


def rows_of(counts, K, seed, tail=0, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(sum(counts) + tail, K, generator=g) * sigma
    x[:, ::37] *= 20
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(counts), 0)
    return x.to(torch.bfloat16).to(DEV), off.to(DEV)


def sums(x, w):
    """x [m, K] w^T and its tolerance."""
    X = x.to(F64)
    s = X @ w.T
    mag = X.abs() @ w.abs().T
    e = 2 * X.shape[1] * U * mag + 2.0 ** -35 * X.abs().amax(1, keepdim=True) * w.abs().sum(1)
    return s, e + 1e-38


def check_matmul(x, off, w, y, f32):
    o = off.tolist()
    for g in range(len(o) - 1):
        a, b = o[g], o[g + 1]
        if a == b:
            continue
        s, e = sums(x[a:b], w[g])
        tol = e + (0.0 if f32 else B) * s.abs()
        err = (y[a:b].to(F64) - s).abs()
        assert (err <= tol).all(), (g, float((err / tol).max()))


def check_swiglu(x, off, w, act, f32):
    o, I = off.tolist(), w.shape[1] // 2
    for g in range(len(o) - 1):
        a, b = o[g], o[g + 1]
        if a == b:
            continue
        s, e = sums(x[a:b], w[g])
        gate, up, eg, eu = s[:, :I], s[:, I:], e[:, :I], e[:, I:]
        silu = gate * torch.sigmoid(gate)
        want = silu * up
        tol = 1.1 * eg * up.abs() + silu.abs() * eu + 1.1 * eg * eu + \
            (2.0 ** -18 * (1 + gate.abs() / 16) + (0.0 if f32 else B)) * want.abs() + 1e-36
        err = (act[a:b].to(F64) - want).abs()
        assert (err <= tol).all(), (g, float((err / tol).max()))


CASES = [([1], 128, 128), ([8], 256, 128), ([3], 384, 256), ([9, 0, 1], 256, 384),
         ([0, 2, 0, 0, 5, 8, 16, 17], 512, 256), ([40], 640, 128), ([1] * 8 + [0] * 56, 1024, 128),
         ([130], 128, 256), ([1], 8192, 128), ([2, 33, 1], 2176, 128), ([1] * 30, 256, 1024)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("counts,K,N", CASES)
def test_products(counts, K, N, fmt):
    exp = -3 if fmt == "nv" else 0
    x, off = rows_of(counts, K, K + N)
    st = moe.new_status(DEV)
    m, w = weights(len(counts), N, K, fmt, K, exp)
    for f32 in (False, True):
        check_matmul(x, off, w, moe.fp4_weight_matmul(x, off, m, out_f32=f32, status=st), f32)
    x = (x.float() / K ** 0.5 / (2 if fmt == "mx" else 4)).to(torch.bfloat16)
    m, w = weights(len(counts), 2 * N, K, fmt, K + 1, exp)
    for f32 in (False, True):
        check_swiglu(x, off, w, moe.fp4_weight_swiglu(x, off, m, out_f32=f32, status=st), f32)
    assert int(st.item()) == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("sigma", [1e-35, 1e-20, 1e20, 3e33])
def test_rows_of_every_magnitude(fmt, sigma):
    x, off = rows_of([3, 12], 512, 3, sigma=sigma)
    m, w = weights(2, 128, 512, fmt, 4)
    check_matmul(x, off, w, moe.fp4_weight_matmul(x, off, m, out_f32=True), True)


def test_all_codes_and_scales():
    """Every code under every scale byte, one product each (a unit row)."""
    for fmt in ("mx", "nv"):
        bl = ref.BLOCK[fmt]
        K, N = 128, 256
        scales = np.arange(256) if fmt == "mx" else np.arange(128)
        scales = np.resize(scales, N).astype(np.uint8)
        code = np.resize(np.arange(16), (N, K)).astype(np.uint8)
        byte = np.repeat(scales[:, None], K // bl, 1)
        m = moe.Fp4Matrix(torch.from_numpy(ref.pack(code)).view(1, N, K // 2).to(DEV),
                          torch.from_numpy(ref.place(byte, None, moe.fp4_scales_size(N, K, fmt)))
                          .to(DEV), fmt, 0)
        nan = 255 if fmt == "mx" else 127
        top = 216 if fmt == "mx" else 127               # magnitudes below 2^90
        vals = ref.values(code, np.minimum(byte, top), fmt, 0)
        x = torch.eye(K, dtype=torch.bfloat16, device=DEV)
        off = torch.tensor([0, K], dtype=torch.int32, device=DEV)
        y = moe.fp4_weight_matmul(x, off, m, out_f32=True).double().cpu().numpy()
        ok = scales < top if fmt == "mx" else scales != nan
        # 2^-127 times a code, and what lies below, is within fp32's subnormals
        assert np.allclose(y[:, ok], vals.T[:, ok], rtol=2.0 ** -24, atol=2.0 ** -148)
        assert np.isnan(y[:, scales == nan]).all()


def test_nonfinite_rows():
    x, off = rows_of([4, 20], 256, 6)
    m, w = weights(2, 128, 256, "mx", 7)
    x[1, 5], x[2, 7], x[9, 3] = float("inf"), float("nan"), -float("inf")
    y = moe.fp4_weight_matmul(x, off, m, out_f32=True).to(F64)
    for r in range(24):
        g = 0 if r < 4 else 1
        want = x[r].to(F64) @ w[g].T
        if r in (1, 2, 9):
            zero = w[g][:, {1: 5, 2: 7, 9: 3}[r]] == 0       # inf times 0
            assert torch.isnan(y[r][zero]).all()
            assert torch.equal(torch.isnan(y[r]), torch.isnan(want))
            assert torch.equal(y[r][torch.isinf(want)], want[torch.isinf(want)])
        else:
            assert torch.isfinite(y[r]).all()


def test_rows_behind_the_last_group_and_of_others():
    x, off = rows_of([2, 0, 3], 256, 8, tail=6)
    m, _ = weights(3, 128, 256, "nv", 9)
    want = moe.fp4_weight_matmul(x, off, m)
    x[5:] = float("nan")
    x[0] = float("nan")
    out = torch.full((11, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got = moe.fp4_weight_matmul(x, off, m, out=out)
    assert got is out and (out[5:] == 7.0).all()
    assert torch.equal(out[1:5], want[1:5])


@pytest.mark.parametrize("off", [[0, 5, 3], [-1, 4, 8], [0, 4, 9]])
def test_bad_offsets(off):
    x, _ = rows_of([4, 4], 128, 10)
    m, _ = weights(2, 128, 128, "mx", 11)
    st = moe.new_status(DEV)
    out = torch.full((8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.fp4_weight_matmul(x, torch.tensor(off, dtype=torch.int32, device=DEV), m, out=out,
                          status=st)
    assert int(st.item()) == moe.DEV_BAD_OFFSETS and (out == 7.0).all()


def test_no_rows():
    m, _ = weights(2, 256, 128, "mx", 12)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    assert moe.fp4_weight_matmul(x, off, m).shape == (0, 256)
    assert moe.fp4_weight_swiglu(x, off, m).shape == (0, 128)
    x = torch.randn((5, 128), device=DEV).to(torch.bfloat16)
    out = torch.full((5, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    assert (moe.fp4_weight_matmul(x, off, m, out=out) == 7.0).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_decoding_step(fmt):
    """A token through routing, the 4-bit FFN and the weighted sum; the FFN
    bit for bit its two products."""
    T, H, I, E, k = 3, 256, 384, 16, 4
    g = torch.Generator().manual_seed(13)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    idx, tw = moe.gate_topk(torch.randn(T, E, generator=g).to(DEV), k)
    w13 = (torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).to(torch.bfloat16).to(DEV)
    w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).to(torch.bfloat16).to(DEV)
    q13, q2 = (moe.fp4_quantize(t, fmt, scale_exp=-4 if fmt == "nv" else 0) for t in (w13, w2))
    r = moe.init_routing(idx, x, E)
    act, y = moe.fp4_weight_mlp(r["expanded_x"], r["offsets"], q13, q2)
    assert torch.equal(act, moe.fp4_weight_swiglu(r["expanded_x"], r["offsets"], q13))
    assert torch.equal(y, moe.fp4_weight_matmul(act, r["offsets"], q2))
    out = moe.finalize_routing(y, r["row_idx"], tw, out_f32=True)
    v13, v2 = moe.fp4_dequantize(q13).to(F64), moe.fp4_dequantize(q2).to(F64)
    want = torch.zeros(T, H, dtype=F64, device=DEV)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            s = v13[e] @ x[t].to(F64)
            want[t] += float(tw[t, j]) * (v2[e] @ (torch.nn.functional.silu(s[:I]) * s[I:]))
    # act and y are rounded to bf16 on the way
    assert float((out.to(F64) - want).norm() / want.norm()) <= 2 * B / 3 ** 0.5


def test_captured_replayed_and_on_another_stream():
    x, off = rows_of([3, 0, 9, 1], 2048, 14)
    m, _ = weights(4, 256, 2048, "mx", 15)
    want = moe.fp4_weight_swiglu(x, off, m)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = moe.fp4_weight_swiglu(x, off, m)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(want, other)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = moe.fp4_weight_swiglu(x, off, m)
    cap.zero_()
    g.replay()
    assert torch.equal(want, cap)
    x.copy_(x.roll(3, 0))
    off.copy_(torch.tensor([0, 0, 1, 13, 13], dtype=torch.int32))
    want = moe.fp4_weight_swiglu(x, off, m)
    for _ in range(3):
        g.replay()
    assert torch.equal(want, cap)


def test_weights_just_written():
    """The products start on the weights before the rows are converted, but not
    before what is in front of the call has ended."""
    x, off = rows_of([1, 2], 4096, 16)
    m, _ = weights(2, 1024, 4096, "mx", 17)
    other, _ = weights(2, 1024, 4096, "mx", 18)
    want = [moe.fp4_weight_matmul(x, off, t) for t in (m, other)]
    buf = moe.Fp4Matrix(torch.zeros_like(m.q), torch.zeros_like(m.sf), "mx", 0)
    for i in range(20):
        src = (m, other)[i & 1]
        buf.q.copy_(src.q)
        buf.sf.copy_(src.sf)
        assert torch.equal(moe.fp4_weight_matmul(x, off, buf), want[i & 1])
