"""The router's training operators on thousands of sequences, against float64
on the GPU (tolerances as in test_gpu_router_grad.py).
"""
import numpy as np
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from tests.test_gpu_router_grad import DEV, U

pytestmark = pytest.mark.gpu


def bounds(T, S, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "even":                       # with fewer tokens than sequences: empty ones between
        b = np.arange(S + 1, dtype=np.int64) * T // S
    elif kind == "ragged":                   # tokens before the first and behind the last one
        b = np.sort(rng.integers(T // 10, T - T // 10, S + 1))
    else:                                    # nearly all empty, at one token in the middle
        b = np.full(S + 1, T // 2)
        b[:4] = [1, 2, 40, T // 3]
        b[-3:] = [T // 2 + 1, T - 7, T - 1]
    return torch.from_numpy(b.astype(np.int32)).to(DEV)


def reference(lg, idx, keep, seq, coef):
    """loss, counts, means, tokens and the loss's gradient with its scale."""
    T, E = lg.shape
    k, S = idx.shape[1], seq.numel() - 1
    b = seq.long()
    t = torch.arange(T, device=DEV)
    sid = torch.searchsorted(b[1:].contiguous(), t, right=True)
    on = keep & (t >= b[0]) & (t < b[-1])
    sid = sid.clamp(max=S - 1)
    p = torch.softmax(lg.double(), 1) * on[:, None]
    n = torch.zeros(S, dtype=torch.int64, device=DEV).index_add_(0, sid, on.long())
    c = torch.zeros(S * E, dtype=torch.int64, device=DEV)
    c.index_add_(0, (sid[:, None] * E + idx.long()).reshape(-1),
                 on[:, None].expand(T, k).reshape(-1).long())
    c = c.view(S, E).double()
    n1 = n.clamp(min=1).double()
    P = torch.zeros((S, E), dtype=torch.float64, device=DEV).index_add_(0, sid, p) / n1[:, None]
    a = coef * E / (k * int((n > 0).sum()))
    loss = a * ((c * P).sum(1) / n1).sum()
    f = (a / (n1 * n1))[sid][:, None]
    pc = (p * c[sid]).sum(1, keepdim=True)
    return loss, c, P, n, f * p * (c[sid] - pc), f * p * (c[sid] + pc)


@pytest.mark.parametrize("kind", ["even", "ragged", "piled"])
@pytest.mark.parametrize("T,E,k,S", [(20000, 64, 4, 8192), (30001, 33, 3, 65536), (70000, 160, 6, 65536),
                                     (5000, 8, 2, 4097), (3000, 600, 2, 5000)])
def test_thousands_of_sequences(T, E, k, S, kind):
    g = torch.Generator(device=DEV).manual_seed(T + S)
    lg = torch.randn((T, E), generator=g, device=DEV) * 1.5
    idx = lg.topk(k, dim=1).indices.to(torch.int32)
    keep = torch.rand(T, generator=g, device=DEV) >= 0.1
    seq = bounds(T, S, kind, 5)
    st = moe.new_status(DEV)
    args = dict(token_mask=keep, seq_offsets=seq, status=st)
    b = moe.balance_loss(lg, idx, 0.5, **args)
    d = moe.gate_topk_backward(lg, idx, balance=b, **args)
    assert int(st.item()) == 0
    loss, c, P, n, ex, sc = reference(lg, idx, keep, seq, 0.5)
    assert torch.equal(b["counts"].double(), c) and torch.equal(b["n_tokens"].long(), n)
    assert ((b["prob_mean"].double() - P).abs() <= (1100 + E / 4) * U * P).all()
    assert abs(float(b["loss"]) - float(loss)) <= (2200 + E) * U * float(loss)
    assert ((d.double() - ex).abs() <= (E + 64) * U * sc + 1e-38).all()


def test_time_does_not_grow_with_the_square_of_the_sequences():
    """65536 sequences, nearly all empty at one token: their outputs are 4096
    times those of 16 sequences, and the pass takes some 20 times as long; with
    a step per sequence and token group, or the bounds read once per sequence,
    it takes 900 times as long.  The limit lies between, at 100."""
    T, E, k = 65536, 64, 6
    lg = torch.randn((T, E), device=DEV)
    idx = lg.topk(k, dim=1).indices.to(torch.int32)

    def shortest(S):
        seq = bounds(T, S, "piled", 1)
        best = float("inf")
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            bal = moe.balance_loss(lg, idx, seq_offsets=seq)
            moe.gate_topk_backward(lg, idx, balance=bal, seq_offsets=seq)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    assert shortest(65536) <= 100 * shortest(16)
