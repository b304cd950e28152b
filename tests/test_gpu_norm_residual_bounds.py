"""norm_residual and its backward pass under bounds that do not ascend inside the
rows: the status word says so and every output buffer keeps what it held, those of
the column sums (whose kernel judges the bounds by itself, for few sequences and for
many) among them.
"""
import ctypes

import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from .test_gpu_norm_residual import BF, DEV, F32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seq", [[0, 5, 3], [-1, 4, 8], [0, 4, 9], [0] * 18 + [9, 8], [-1] + [2] * 20])
def test_bad_bounds_leave_every_buffer(seq):
    T, H, S = 8, 264, len(seq) - 1
    d = make(T, H, None, 31)
    gate = torch.randn(S, H, generator=torch.Generator().manual_seed(32)).to(BF).to(DEV)
    off = torch.tensor(seq, dtype=torch.int32, device=DEV)
    L, p = moe.lib(), lambda t: ctypes.c_void_p(t.data_ptr())            # noqa: E731
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    st = moe.new_status(DEV)
    mark = lambda *shape, t=F32: torch.full(shape, 7.0, dtype=t, device=DEV)   # noqa: E731
    r, xn, kp, kn = mark(T, H, t=BF), mark(T, H, t=BF), mark(T), mark(T)
    assert L.moe_norm_residual(p(d["x"]), p(d["y"]), p(d["gp"]), p(gate), p(off), S, p(d["gn"]), T, H, 1.0, 1e-6,
                               moe.POST_NORM, p(r), p(xn), p(kp), p(kn), p(st), s) == 0
    assert int(st.item()) == moe.DEV_BAD_OFFSETS
    for t in (r, xn, kp, kn):
        assert (t == 7.0).all()
    st.zero_()
    d_x, d_y, d_gp, d_gate, d_gn = mark(T, H, t=BF), mark(T, H, t=BF), mark(H), mark(S, H), mark(H)
    n = moe.norm_residual_backward_workspace_size(T, H, S)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    assert L.moe_norm_residual_backward(p(d["d_r"]), p(d["d_xn"]), p(d["y"]), p(d["x"]), p(kp), p(kn), p(d["gp"]),
                                        p(gate), p(off), S, p(d["gn"]), T, H, 1.0, moe.POST_NORM, p(d_x), p(d_y),
                                        p(d_gp), p(d_gate), p(d_gn), p(ws), n, p(st), s) == 0
    assert int(st.item()) == moe.DEV_BAD_OFFSETS
    for t in (d_x, d_y, d_gp, d_gate, d_gn):
        assert (t == 7.0).all()
