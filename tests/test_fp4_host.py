"""4-bit operands and the router's training operators, what needs no GPU: the
scale layout, the rounding argument of the 16-column format, and the refusals
of the C entry points and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from tests import _fp4_ref as ref


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


P = ctypes.c_void_p
FAKE = P(0x1000)


def mat(q=0x1000, sf=0x1000, fmt=0, exp=0):
    return ctypes.byref(moe._Fp4(q, sf, fmt, exp))


def test_reference_scale_rounding_matches_torch():
    v = np.concatenate([np.linspace(0, 500, 4001), 2.0 ** np.linspace(-12, 9, 3001),
                        (np.arange(1, 256) * 2.0 ** -12)])
    r, byte = ref.e4m3_round(v)
    t = torch.from_numpy(v).clamp(max=448.0).to(torch.float32).to(torch.float8_e4m3fn)
    f32 = torch.from_numpy(v).to(torch.float32).double().numpy() == v
    assert np.array_equal(r[f32], t.double().numpy()[f32])
    assert np.array_equal(byte[f32], t.view(torch.uint8).numpy()[f32])


@pytest.mark.parametrize("sizes", [[0], [1], [128, 128], [127, 1, 0, 300, 129], [5] * 40,
                                   [0, 0, 1000, 0]])
def test_scale_blocks_of_groups_do_not_overlap(sizes):
    off = np.concatenate([[0], np.cumsum(sizes)])
    n, G = int(off[-1]), len(sizes)
    blk, loc = ref.row_blocks(n, off)
    at = blk * 128 + loc
    assert len(set(at.tolist())) == n and (at >= 0).all()
    # a group's blocks are its own, inside the size the library asks for
    for g in range(G):
        mine = set(blk[off[g]:off[g + 1]].tolist())
        assert not mine & set(np.delete(blk, np.arange(off[g], off[g + 1])).tolist())
    for fmt, nb in (("mx", 4), ("nv", 8)):
        if n:
            assert ref.scale_positions(n, nb, off).max() < moe.fp4_scales_size(n, 128, fmt, G)


def test_scales_size(L):
    assert moe.fp4_scales_size(128, 256, "mx") == 2 * 512
    assert moe.fp4_scales_size(129, 256, "nv") == 2 * 4 * 512
    assert moe.fp4_scales_size(129, 256, "nv", groups=3) == 4 * 4 * 512
    assert moe.fp4_scales_size(0, 128, "mx") == 0
    n = ctypes.c_size_t()
    assert L.moe_fp4_scales_size(4, 192, 0, 0, ctypes.byref(n)) == 2
    assert L.moe_fp4_scales_size(4, 128, 2000, 0, ctypes.byref(n)) == 2
    assert L.moe_fp4_scales_size(4, 128, 0, 2, ctypes.byref(n)) == 1
    assert L.moe_fp4_scales_size(-1, 128, 0, 0, ctypes.byref(n)) == 1
    assert L.moe_fp4_scales_size(4, 128, 0, 0, None) == 1


def test_quotients_are_midpoints_or_far_from_them():
    """The NV rounding argument: bf16 value / e4m3 scale is exactly a midpoint
    of the e2m1 grid or at least 2^-8 away from every one, relative to it, so
    an error of 2^-22 before rounding to 13 bits changes no code."""
    x = np.arange(128, 256, dtype=np.float64)                 # 8 significant bits
    s = np.concatenate([np.arange(8, 16), np.arange(1, 8)]).astype(np.float64)
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for e in range(-12, 4):
        qt = (x[:, None] / s[None, :]) * 2.0 ** e
        d = np.abs(qt[:, :, None] / mid - 1.0)
        # exactness decided on integers: x 2^e == mid s
        tie = (x[:, None, None] * 2.0 ** e) == (s[None, :, None] * mid)
        assert (d[~tie] >= 2.0 ** -8).all()
        # the kernel's steps in fp32: times the rounded reciprocal, then 13 bits
        y = (x[:, None].astype(np.float32) * np.float32(2.0 ** e)) * \
            (np.float32(1.0) / s[None, :].astype(np.float32))
        y = ((y.view(np.uint32) + np.uint32(0x400)) & np.uint32(0xFFFFF800)).view(np.float32)
        y3 = np.broadcast_to(y[:, :, None].astype(np.float64), tie.shape)
        m3 = np.broadcast_to(mid, tie.shape)
        assert (y3[tie] == m3[tie]).all()
        q3 = np.broadcast_to(qt[:, :, None], tie.shape)
        assert ((y3 > m3)[~tie] == (q3 > m3)[~tie]).all()


def test_refusals_of_the_products(L):
    mm, sw, mlp = L.moe_fp4_grouped_matmul, L.moe_fp4_grouped_swiglu, L.moe_fp4_grouped_mlp
    ok = dict(n=4, K=128, N=128)

    def m(a=None, off=FAKE, G=2, w=None, n=4, K=128, N=128, y=FAKE):
        return mm(a or mat(), off, G, w or mat(), n, K, N, 0, y, None, None)
    assert m(K=192) == 2 and m(N=64) == 2 and m(G=2000) == 2
    assert m(K=0) == 1 and m(n=-1) == 1 and m(G=0) == 1 and m(N=0) == 1
    assert m(a=mat(fmt=0), w=mat(fmt=1)) == 1                  # one format per call
    assert m(a=mat(fmt=3), w=mat(fmt=3)) == 1
    assert m(a=mat(exp=1), w=mat()) == 1                       # mx carries no exponent
    assert m(a=mat(fmt=1, exp=61), w=mat(fmt=1)) == 1
    assert m(off=None) == 1 and m(y=None) == 1 and m(y=P(0x1008)) == 1
    assert m(w=mat(q=None)) == 1 and m(w=mat(sf=0x1008)) == 1 and m(a=mat(q=0x1001)) == 1
    assert m(n=0, y=None, a=mat(q=None, sf=None)) == 0         # nothing to do
    assert mm(None, FAKE, 2, mat(), 4, 128, 128, 0, FAKE, None, None) == 1
    # sizes whose tile numbers pass 32 bits
    assert m(n=2 ** 30, K=1 << 19, N=128) == 2
    assert m(n=2 ** 31 - 1) == 2 and m(K=1 << 21) == 2
    # swiglu: exactly one form of the result
    assert sw(mat(), FAKE, 2, mat(), 4, 128, 128, None, None, None, None) == 1
    assert sw(mat(), FAKE, 2, mat(), 4, 128, 128, FAKE, mat(), None, None) == 1
    assert sw(mat(), FAKE, 2, mat(), 4, 128, 128, None, mat(fmt=1), None, None) == 1
    assert sw(mat(), FAKE, 2, mat(), 4, 128, 128, None, mat(q=None), None, None) == 1
    assert sw(mat(), FAKE, 2, mat(), 4, 128, 96, FAKE, None, None, None) == 2
    # the factors of swiglu's two operands together
    assert sw(mat(fmt=1, exp=40), FAKE, 2, mat(fmt=1, exp=30), 4, 128, 128, FAKE, None, None,
              None) == 2
    assert mlp(mat(fmt=1, exp=-40), FAKE, 2, mat(fmt=1, exp=-30), mat(fmt=1), 4, 128, 128, 0,
               mat(fmt=1), FAKE, None, None) == 2
    # mlp
    assert mlp(mat(), FAKE, 2, mat(), mat(), 4, 128, 128, 0, None, FAKE, None, None) == 1
    assert mlp(mat(), FAKE, 2, mat(), mat(fmt=1), 4, 128, 128, 0, mat(), FAKE, None, None) == 1
    assert mlp(mat(), FAKE, 2, mat(), mat(), 4, 128, 128, 0, mat(), None, None, None) == 1
    assert mlp(mat(), FAKE, 2, mat(), mat(), 4, 128, 192, 0, mat(), FAKE, None, None) == 2
    assert ok


def test_refusals_of_the_conversions(L):
    q, d = L.moe_fp4_quantize, L.moe_fp4_dequantize
    assert q(FAKE, 4, 192, None, 1, None, 0, mat(), None, None) == 2
    assert q(FAKE, 4, 1 << 21, None, 1, None, 0, mat(), None, None) == 2
    assert q(FAKE, 4, 128, None, 2, None, 0, mat(), None, None) == 2       # k needs rows
    assert q(FAKE, 4, 128, FAKE, 33, None, 0, mat(), None, None) == 2
    assert q(FAKE, 4, 128, FAKE, 2, None, 3, mat(), None, None) == 1       # groups need offsets
    assert q(FAKE, 4, 128, FAKE, 2, FAKE, 0, mat(), None, None) == 1
    assert q(FAKE, 4, 128, FAKE, 2, FAKE, 1025, mat(), None, None) == 2
    assert q(P(0x1004), 4, 128, None, 1, None, 0, mat(), None, None) == 1
    assert q(FAKE, 4, 128, None, 1, None, 0, mat(exp=2), None, None) == 1
    assert q(FAKE, 4, 128, None, 1, None, 0, None, None, None) == 1
    assert q(FAKE, -4, 128, None, 1, None, 0, mat(), None, None) == 1
    assert q(FAKE, 2 ** 30, 128, FAKE, 2, None, 0, mat(), None, None) == 2  # T k past 31 bits
    assert q(None, 0, 128, None, 1, None, 0, mat(q=None, sf=None), None, None) == 0
    assert d(mat(), 4, 192, None, 0, FAKE, None) == 2
    assert d(mat(), 4, 128, None, 1, FAKE, None) == 1
    assert d(mat(), 4, 128, None, 0, None, None) == 1
    assert d(None, 4, 128, None, 0, FAKE, None) == 1
    assert d(mat(q=None, sf=None), 0, 128, None, 0, None, None) == 0


def test_refusals_of_the_router_operators(L):
    n = ctypes.c_size_t()
    assert L.moe_balance_loss_workspace_size(100, 8, 1, ctypes.byref(n)) == 0 and n.value > 0
    assert L.moe_balance_loss_workspace_size(100, 2000, 1, ctypes.byref(n)) == 2
    assert L.moe_balance_loss_workspace_size(100, 8, 0, ctypes.byref(n)) == 1
    assert L.moe_balance_loss_workspace_size(100, 8, 65537, ctypes.byref(n)) == 2
    assert L.moe_balance_loss_workspace_size(2 ** 30 + 1, 8, 1, ctypes.byref(n)) == 2
    L.moe_balance_loss_workspace_size(100, 8, 2, ctypes.byref(n))
    bl = L.moe_balance_loss

    def f(lg=FAKE, idx=FAKE, seq=FAKE, S=2, T=100, E=8, k=2, loss=FAKE, ws=FAKE, size=n.value):
        return bl(lg, idx, None, seq, S, T, E, k, 1.0, loss, FAKE, FAKE, FAKE, ws, size, None, None)
    assert f(k=9) == 2 and f(E=1025) == 2 and f(T=-1) == 1 and f(k=0) == 1
    assert f(seq=None) == 1                                    # two sequences need bounds
    assert f(lg=None) == 1 and f(idx=None) == 1 and f(loss=None) == 1
    assert f(size=n.value - 1) == 3 and f(ws=None) == 3 and f(ws=P(0x1010)) == 3
    tb = L.moe_gate_topk_backward

    def b(lg=FAKE, idx=FAKE, dw=FAKE, seq=None, S=1, c=FAKE, nt=FAKE, T=4, E=8, k=2, d=FAKE):
        return tb(lg, idx, dw, None, seq, S, c, nt, None, 1.0, T, E, k, 0, d, None, None)
    assert b(k=9) == 2 and b(E=1025) == 2 and b(T=-1) == 1 and b(T=2 ** 30 + 1, k=1) == 2
    assert b(S=65537, seq=FAKE) == 2
    assert b(c=None) == 1 and b(nt=None) == 1                  # both or neither
    assert b(S=2) == 1 and b(S=0) == 1
    assert b(lg=None) == 1 and b(d=None) == 1 and b(idx=None) == 1
    assert b(T=0, lg=None, d=None) == 0
    fb = L.moe_finalize_routing_backward

    def r(do=FAKE, y=FAKE, rows=FAKE, w=FAKE, T=4, H=64, k=2, dy=FAKE, dw=FAKE):
        return fb(do, y, rows, w, T, H, k, 0, dy, dw, None, None)
    assert r(H=12) == 2 and r(k=33) == 2 and r(T=-1) == 1 and r(k=0) == 1
    assert r(do=None) == 1 and r(y=None) == 1 and r(rows=None) == 1 and r(w=None) == 1
    assert r(dy=None) == 1 and r(dw=None) == 1 and r(dy=P(0x1008)) == 1 and r(y=P(0x1002)) == 1
    assert r(T=0, do=None) == 0


def test_valid_calls_without_a_gpu_fail_loudly(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    n = ctypes.c_size_t()
    L.moe_balance_loss_workspace_size(4, 8, 1, ctypes.byref(n))
    assert L.moe_balance_loss(FAKE, FAKE, None, None, 1, 4, 8, 2, 1.0, FAKE, FAKE, FAKE, FAKE, FAKE,
                              n.value, None, None) == 5
    assert L.moe_gate_topk_backward(FAKE, FAKE, FAKE, None, None, 1, None, None, None, 0.0, 4, 8, 2,
                                    0, FAKE, None, None) == 5
    assert L.moe_finalize_routing_backward(FAKE, FAKE, FAKE, FAKE, 4, 64, 2, 0, FAKE, FAKE, None,
                                           None) == 5
    assert L.moe_fp4_quantize(FAKE, 4, 128, None, 1, None, 0, mat(), None, None) == 5
    assert L.moe_fp4_dequantize(mat(), 4, 128, None, 0, FAKE, None) == 5
    assert L.moe_fp4_grouped_matmul(mat(), FAKE, 2, mat(), 4, 128, 128, 0, FAKE, None, None) == 5


def test_the_binding_refuses_wrong_tensors():
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    lg, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32)
    with pytest.raises(TypeError):
        moe.balance_loss(lg.double(), idx)
    with pytest.raises(TypeError):
        moe.balance_loss(lg, idx.long())
    with pytest.raises(ValueError):
        moe.balance_loss(lg, idx, token_mask=torch.zeros(5, dtype=torch.bool))
    with pytest.raises(TypeError):
        moe.balance_loss(lg, idx, token_mask=torch.zeros(4, dtype=f32))
    with pytest.raises(ValueError):
        moe.balance_loss(lg, idx, seq_offsets=torch.zeros(1, dtype=i32))
    with pytest.raises(ValueError):
        moe.gate_topk_backward(lg, idx, torch.zeros(4, 3))
    bal = dict(counts=torch.zeros(2, 8, dtype=i32), n_tokens=torch.zeros(2, dtype=i32), coef=1.0)
    with pytest.raises(ValueError):
        moe.gate_topk_backward(lg, idx, balance=bal)           # another number of sequences
    with pytest.raises(ValueError):
        moe.finalize_routing_backward(torch.zeros(4, 64), torch.zeros(7, 64), idx.view(-1),
                                      torch.zeros(4, 2))
    m = moe.Fp4Matrix(torch.zeros(4, 64, dtype=u8), torch.zeros(100, dtype=u8))
    w = moe.Fp4Matrix(torch.zeros(2, 128, 64, dtype=u8), torch.zeros(1024, dtype=u8))
    off = torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError):
        moe.fp4_grouped_matmul(m, torch.zeros(2, dtype=i32), w)
    with pytest.raises(ValueError):
        moe._fp4_arg(m, "a", 2, m.q.device)                     # scales too small
    with pytest.raises(ValueError):
        moe.fp4_grouped_matmul(moe.Fp4Matrix(torch.zeros(4, 128, dtype=u8), m.sf), off, w)
    with pytest.raises(ValueError):
        moe.fp4_quantize(torch.zeros(4, 128, dtype=torch.bfloat16), "int4")
    with pytest.raises(TypeError):
        moe.fp4_quantize(torch.zeros(4, 128))
    with pytest.raises(ValueError):
        moe.fp4_quantize(torch.zeros(4, 128, dtype=torch.bfloat16), k=2)
    with pytest.raises(ValueError):                             # CPU tensors
        moe.fp4_dequantize(moe.Fp4Matrix(torch.zeros(4, 64, dtype=u8),
                                         torch.zeros(512, dtype=u8)))
