"""Refusals of norm_residual and its backward pass, before any CUDA work."""
import ctypes

import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe

P = ctypes.c_void_p
fake, odd = P(0x1000), P(0x1008)
POST = moe.POST_NORM


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


def fwd(L, x=fake, y=fake, gp=fake, gate=fake, seq=fake, S=2, gn=fake, T=4, H=64, flags=POST, r=fake,
        xn=fake, kp=fake, kn=fake):
    return L.moe_norm_residual(x, y, gp, gate, seq, S, gn, T, H, 1.0, 1e-6, flags, r, xn, kp, kn, None,
                               None)


def size(L, T=4, H=64, S=2):
    b = ctypes.c_size_t(0)
    assert L.moe_norm_residual_backward_workspace_size(T, H, S, ctypes.byref(b)) == 0
    return b.value


def bwd(L, d_r=fake, d_xn=fake, y=fake, r=fake, kp=fake, kn=fake, gp=fake, gate=fake, seq=fake, S=2,
        gn=fake, T=4, H=64, flags=POST, d_x=fake, d_y=fake, dgp=fake, dgt=fake, dgn=fake, ws=fake,
        nbytes=None):
    return L.moe_norm_residual_backward(d_r, d_xn, y, r, kp, kn, gp, gate, seq, S, gn, T, H, 1.0, flags,
                                        d_x, d_y, dgp, dgt, dgn, ws,
                                        size(L) if nbytes is None else nbytes, None, None)


@pytest.mark.parametrize("f", [fwd, bwd])
def test_sizes_and_modes(L, f):
    assert f(L, T=-1) == 1 and f(L, H=0) == 1 and f(L, S=0) == 1
    assert f(L, H=68) == 2 and f(L, H=8200) == 2 and f(L, S=65537) == 2 and f(L, T=(1 << 30) + 1) == 2
    assert f(L, seq=None) == 1                       # two sequences without bounds
    assert f(L, flags=0) == 1                        # gamma_post without its norm
    for name in ("y", "gp", "gate", "gn"):
        assert f(L, **{name: odd}) == 1, name
    assert f(L, y=None) == 1


def test_forward_pointers(L):
    for name in ("x", "r"):
        assert fwd(L, **{name: None}) == 1 and fwd(L, **{name: odd}) == 1
    assert fwd(L, xn=odd) == 1
    assert fwd(L, xn=None) == 1 and fwd(L, xn=None, gn=None) == 1      # rstd_next of no norm
    assert fwd(L, T=0, x=None, y=None, r=None) == 0


def test_backward_pointers(L):
    for name in ("d_r", "d_xn", "r", "d_x", "d_y"):
        assert bwd(L, **{name: odd}) == 1, name
    assert bwd(L, r=None) == 1 and bwd(L, kp=None) == 1 and bwd(L, kn=None) == 1
    assert bwd(L, d_xn=None) == 1                    # d_gamma_next of no norm
    assert bwd(L, d_xn=None, d_r=None, gn=None, dgn=None) == 1
    assert bwd(L, gate=None) == 1                    # d_gate of no gate
    assert bwd(L, ws=None) == 3 and bwd(L, ws=P(0x1010)) == 3 and bwd(L, nbytes=size(L) - 1) == 3
    b = ctypes.c_size_t(0)
    assert L.moe_norm_residual_backward_workspace_size(4, 60, 1, ctypes.byref(b)) == 2
    assert L.moe_norm_residual_backward_workspace_size(4, 64, 1, None) == 1


def test_binding_refuses():
    bf = torch.bfloat16
    x, y, g = torch.zeros((4, 64), dtype=bf), torch.zeros((4, 64), dtype=bf), torch.ones(64, dtype=bf)
    gate, seq = torch.ones((2, 64), dtype=bf), torch.tensor([0, 2, 4], dtype=torch.int32)
    saved = dict(r=x, rstd_post=torch.ones(4), rstd_next=torch.ones(4))
    T, V = TypeError, ValueError
    n, b = moe.norm_residual, moe.norm_residual_backward
    for err, f in (
            (T, lambda: n(x.half(), y)), (T, lambda: n(x, y.double())), (V, lambda: n(x[:3], y)),
            (V, lambda: n(x[0], y[0])), (T, lambda: n(x, y, gamma_post=g.float())),
            (V, lambda: n(x, y, gamma_post=g[:32])), (V, lambda: n(x, y, gamma_next=g, next_norm=False)),
            (V, lambda: n(x, y, gamma_post=g, post_norm=False)), (T, lambda: n(x, y, gate=gate.float())),
            (V, lambda: n(x, y, gate=gate)), (V, lambda: n(x, y, gate=gate, seq_offsets=seq[:2])),
            (T, lambda: n(x, y, gate=gate, seq_offsets=seq.long())), (V, lambda: n(x.t(), y.t())),
            (V, lambda: b(None, None, y, saved)), (T, lambda: b(x.float(), x, y, saved)),
            (T, lambda: b(x, x.float(), y, saved)), (V, lambda: b(x[:2], x, y, saved)),
            (V, lambda: b(x, x, y, dict(saved, rstd_post=torch.ones(3)))),
            (T, lambda: b(x, x, y, dict(saved, rstd_next=torch.ones(4).double())))):
        with pytest.raises(err):
            f()
