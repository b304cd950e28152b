"""Refusals of the products of bf16 rows and 4-bit weights, before any CUDA work."""
import ctypes

import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe

P = ctypes.c_void_p
fake, odd = P(0x1000), P(0x1008)


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


def mat(q=0x1000, sf=0x1000, fmt=0, exp=0):
    return ctypes.byref(moe._Fp4(q, sf, fmt, exp))


def need(L, n, K, N=128, G=4):
    b = ctypes.c_size_t(0)
    assert L.moe_fp4_weight_workspace_size(n, K, N, G, ctypes.byref(b)) == 0
    return b.value


def call(L, which="matmul", x=fake, off=fake, G=4, w=None, n=10, K=128, N=128, out=fake, ws=fake,
         nbytes=None):
    fn = getattr(L, "moe_fp4_weight_" + which)
    return fn(x, off, G, mat() if w is None else w, n, K, N, 0, out, ws,
              need(L, 10, 128) if nbytes is None else nbytes, None, None)


@pytest.mark.parametrize("which", ["matmul", "swiglu"])
def test_products_refuse(L, which):
    c = lambda **k: call(L, which, **k)                                   # noqa: E731
    assert c(G=0) == 1 and c(n=-1) == 1 and c(K=0) == 1 and c(N=-128) == 1
    assert c(G=1025) == 2 and c(K=192) == 2 and c(N=64) == 2 and c(K=1 << 21) == 2
    assert c(w=mat(fmt=2)) == 1 and c(w=mat(exp=1)) == 1 and c(w=mat(fmt=1, exp=61)) == 1
    assert c(w=mat(q=None)) == 1 and c(w=mat(sf=0x1004)) == 1
    for name in ("x", "off", "out"):
        assert c(**{name: None}) == 1, name
    for name in ("x", "out"):
        assert c(**{name: odd}) == 1, name
    assert c(ws=None) == 3 and c(ws=P(0x1010)) == 3 and c(nbytes=need(L, 10, 128) - 1) == 3
    assert c(n=0, x=None, out=None, ws=None) == 0


def test_mlp_refuses(L):
    def c(x=fake, n=10, H=128, I=256, w13=None, w2=None, act=fake, y=fake, nbytes=None):
        return L.moe_fp4_weight_mlp(x, fake, 4, w13 or mat(), w2 or mat(), n, H, I, 0, act, y, fake,
                                    max(need(L, 10, 256), need(L, 10, 128, 256))
                                    if nbytes is None else nbytes, None, None)
    assert c(H=100) == 2 and c(I=100) == 2
    assert c(w2=mat(fmt=3)) == 1 and c(w13=mat(exp=2)) == 1
    assert c(x=None) == 1 and c(act=None) == 1 and c(y=odd) == 1
    assert c(nbytes=max(need(L, 10, 256), need(L, 10, 128, 256)) - 1) == 3    # the larger one counts
    assert c(n=0, x=None, act=None, y=None) == 0


def test_workspace_size(L):
    b = ctypes.c_size_t(0)
    assert L.moe_fp4_weight_workspace_size(3, 100, 128, 1, ctypes.byref(b)) == 2
    assert L.moe_fp4_weight_workspace_size(3, 128, 100, 1, ctypes.byref(b)) == 2
    assert L.moe_fp4_weight_workspace_size(-1, 128, 128, 1, ctypes.byref(b)) == 1
    assert L.moe_fp4_weight_workspace_size(3, 128, 128, 0, ctypes.byref(b)) == 1
    assert L.moe_fp4_weight_workspace_size(3, 128, 128, 1, None) == 1
    assert need(L, 3, 128) >= 12 * 3 * 64 + 3 * 4


def test_binding_refuses():
    w = moe.Fp4Matrix(torch.zeros((2, 256, 64), dtype=torch.uint8),
                      torch.zeros(moe.fp4_scales_size(512, 128, "mx"), dtype=torch.uint8), "mx", 0)
    x, off = torch.zeros((3, 128), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    T, V = TypeError, ValueError
    short = moe.Fp4Matrix(w.q, w.sf[:-1], "mx", 0)
    for f in (moe.fp4_weight_matmul, moe.fp4_weight_swiglu):
        for err, a in ((T, (x.float(), off, w)), (T, (x, off.long(), w)), (V, (x, off[:2], w)),
                       (V, (x[:, :64], off, w)), (V, (x[0], off, w)), (V, (x, off, short)),
                       (V, (x.t(), off, w))):
            with pytest.raises(err):
                f(*a)
        with pytest.raises(T):
            f(x, off, w, out=torch.zeros((3, 256)))
        with pytest.raises(V):
            f(x, off, w, out=torch.zeros((3, 64), dtype=torch.bfloat16))
    with pytest.raises(V):
        moe.fp4_weight_mlp(x, off, w, w)
