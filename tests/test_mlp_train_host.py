"""Refusals of the expert FFN's training passes, all before any CUDA work."""
import ctypes

import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe

P = ctypes.c_void_p
fake = P(0x1000)
odd = P(0x1008)


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


def fwd(L, x=fake, off=fake, G=4, w13=fake, w2=fake, n=10, H=128, I=128, h=fake, act=fake, y=fake):
    return L.moe_grouped_mlp_train(x, off, G, w13, w2, n, H, I, h, act, y, None, None)


def bwd(L, d_y=fake, x=fake, off=fake, G=4, h=fake, w13=fake, w2=fake, n=10, H=128, I=128, flags=0,
        d_x=fake, d_w13=fake, d_w2=fake, ws=fake, nbytes=None):
    if nbytes is None:
        b = ctypes.c_size_t(0)
        L.moe_grouped_mlp_backward_workspace_size(max(n, 0), 128, ctypes.byref(b))
        nbytes = b.value
    return L.moe_grouped_mlp_backward(d_y, x, off, G, h, w13, w2, n, H, I, flags, d_x, d_w13, d_w2,
                                      ws, nbytes, None, None)


def test_sizes(L):
    for f in (fwd, bwd):
        assert f(L, G=0) == 1 and f(L, n=-1) == 1 and f(L, H=0) == 1 and f(L, I=-128) == 1
        assert f(L, G=1025) == 2 and f(L, H=192) == 2 and f(L, I=96) == 2
        assert f(L, H=1 << 21) == 2 and f(L, I=1 << 20) == 2 and f(L, n=2 ** 31 - 1) == 2


def test_pointers(L):
    for name in ("x", "off", "w13", "w2", "h", "act", "y"):
        assert fwd(L, **{name: None}) == 1, name
    for name in ("x", "w13", "w2", "h", "act", "y"):
        assert fwd(L, **{name: odd}) == 1, name
    for name in ("d_y", "x", "off", "h", "w13", "w2"):
        assert bwd(L, **{name: None}) == 1, name
    for name in ("d_y", "x", "h", "w13", "w2", "d_x", "d_w13", "d_w2"):
        assert bwd(L, **{name: odd}) == 1, name


def test_workspace_and_flags(L):
    b = ctypes.c_size_t(0)
    assert L.moe_grouped_mlp_backward_workspace_size(10, 128, ctypes.byref(b)) == 0
    assert b.value >= 10 * 3 * 128 * 2
    assert L.moe_grouped_mlp_backward_workspace_size(10, 100, ctypes.byref(b)) == 2
    assert L.moe_grouped_mlp_backward_workspace_size(10, 128, None) == 1
    assert bwd(L, nbytes=b.value - 1) == 3
    assert bwd(L, ws=None) == 3 and bwd(L, ws=P(0x1010)) == 3
    # adding is for fp32 buffers
    assert bwd(L, flags=moe.DW_ACCUMULATE) == 1
    # nothing asked for
    assert bwd(L, d_x=None, d_w13=None, d_w2=None) == 0


def test_no_rows_need_no_rows_pointers(L):
    assert fwd(L, n=0, x=None, h=None, act=None, y=None) == 0


def test_binding_refuses():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    w13, w2 = torch.zeros((2, 256, 128), dtype=torch.bfloat16), \
        torch.zeros((2, 128, 128), dtype=torch.bfloat16)
    h, d_y = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros_like(x)
    T, V = TypeError, ValueError
    for err, f in (
            (T, lambda: moe.grouped_mlp_train(x.float(), off, w13, w2)),
            (T, lambda: moe.grouped_mlp_train(x, off.long(), w13, w2)),
            (V, lambda: moe.grouped_mlp_train(x, off[:2], w13, w2)),
            (V, lambda: moe.grouped_mlp_train(x, off, w13[:, :128], w2)),
            (V, lambda: moe.grouped_mlp_train(x.t(), off, w13, w2)),
            (V, lambda: moe.grouped_mlp_train(x[0], off, w13, w2)),
            (V, lambda: moe.grouped_mlp_backward(d_y[:3], x, off, h, w13, w2)),
            (V, lambda: moe.grouped_mlp_backward(d_y, x, off, h[:, :128], w13, w2)),
            (T, lambda: moe.grouped_mlp_backward(d_y.float(), x, off, h, w13, w2)),
            (V, lambda: moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, need=("w3",))),
            (V, lambda: moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, accumulate=True)),
            (V, lambda: moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=True,
                                                 accumulate=True)),
            (T, lambda: moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=True,
                                                 d_w13=w13.clone())),
            (T, lambda: moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, d_w2=w2.float()))):
        with pytest.raises(err):
            f()
