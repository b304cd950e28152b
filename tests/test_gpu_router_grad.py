"""The router's training operators against float64 on the CPU.

Tolerances: probabilities and everything linear in them carry a few fp32
roundings (exp, the sum of E terms, the products): relative 2^-24 per step.
 prob_mean: (E / 4 + 40) 2^-24 relative per probability, plus the sum over a
   sequence in pieces (at most 64 + 1024 additions in a row): 1100 2^-24 in
   all covers both.
 gradients: each term is a product of at most 6 such factors against the row's
   scale: (E + 64) 2^-24 of scale * p * (c + sum p c) for the balance term and
   of |w| (|dw| + sum |w dw|) for the weights'.
 dot products over H: one fp32 step per addition, H 2^-24 sum |d y|.
"""
import numpy as np
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def softmax(z):
    m = z.max(axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(z - m)
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def ref_balance(lg, idx, coef, keep, seq):
    E, k = lg.shape[1], idx.shape[1]
    S = len(seq) - 1
    c, P, n = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    total = 0.0
    for s in range(S):
        t = np.arange(seq[s], seq[s + 1])
        t = t[keep[t]]
        n[s] = len(t)
        if not len(t):
            continue
        for e in idx[t].reshape(-1):
            if 0 <= e < E:
                c[s, e] += 1
        P[s] = softmax(lg[t]).mean(axis=0)
        total += E / (k * len(t)) * (c[s] * P[s]).sum()
    live = max((n > 0).sum(), 1)
    return coef * total / live, c, P, n


def ref_grad(lg, idx, dw, renorm, keep, coef, seq, c, n, d_loss):
    """-> gradient and its tolerance's scale."""
    T, E = lg.shape
    k = idx.shape[1]
    d, tol = np.zeros((T, E)), np.zeros((T, E))
    t = np.nonzero(keep)[0]
    if not len(t):
        return d, tol
    p = softmax(lg[t])
    dd, tt = np.zeros_like(p), np.zeros_like(p)
    if c is not None:
        live = max((n > 0).sum(), 1)
        for s in range(len(seq) - 1):
            m = (t >= seq[s]) & (t < seq[s + 1])
            if not m.any():
                continue
            a = d_loss * coef * E / (k * live * float(n[s]) ** 2)
            pc = (p[m] * c[s]).sum(axis=1, keepdims=True)
            dd[m] += a * p[m] * (c[s] - pc)
            tt[m] += abs(a) * p[m] * (c[s] + pc)
    if dw is not None:
        for r, tok in enumerate(t):
            ii = [(j, e) for j, e in enumerate(idx[tok]) if 0 <= e < E]
            if not ii:
                continue
            js, es = np.array([j for j, _ in ii]), np.array([e for _, e in ii])
            g = dw[tok, js]
            if renorm:
                z = lg[tok, es]
                w = np.exp(z - z.max())
                w /= w.sum()
                np.add.at(dd[r], es, w * (g - (w * g).sum()))
                np.add.at(tt[r], es, w * (np.abs(g) + (w * np.abs(g)).sum()))
            else:
                w = p[r, es]
                dd[r] -= p[r] * (w * g).sum()
                tt[r] += p[r] * (w * np.abs(g)).sum()
                np.add.at(dd[r], es, w * g)
                np.add.at(tt[r], es, w * np.abs(g))
    d[t], tol[t] = dd, tt
    return d, tol


def case(T, E, k, S, pad, seed):
    rng = np.random.default_rng(seed)
    lg = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)
    keep = rng.random(T) >= pad
    seq = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    if S == 1:
        seq[:] = (0, T)
    return rng, lg, idx, keep, seq


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


CASES = [(1, 1, 1, 1, 0.0), (1, 8, 2, 1, 0.0), (64, 8, 2, 1, 0.0), (700, 64, 8, 4, 0.2),
         (1000, 7, 3, 9, 0.5), (513, 160, 6, 3, 0.1), (40, 1024, 32, 2, 0.0),
         (33, 1023, 32, 2, 0.1), (300, 65, 32, 40, 0.3), (5000, 16, 16, 2, 0.05),
         (90, 256, 4, 1, 1.0), (2500, 512, 9, 5, 0.1), (60, 30, 30, 200, 0.0)]


@pytest.mark.parametrize("T,E,k,S,pad", CASES)
@pytest.mark.parametrize("renorm", [True, False])
def test_balance_loss_and_gradient(T, E, k, S, pad, renorm):
    rng, lg, idx, keep, seq = case(T, E, k, S, pad, T + E)
    dw = rng.standard_normal((T, k)).astype(np.float32) * 1e-2
    dev_lg = lg.copy()
    dev_lg[~keep] = np.nan                     # masked places hold anything
    dev_dw = dw.copy()
    dev_dw[~keep] = np.inf
    mask = cu(keep) if pad else None
    seqt = cu(seq) if S > 1 else None
    st = moe.new_status(DEV)
    coef, dl = 0.02, 0.6
    b = moe.balance_loss(cu(dev_lg), cu(idx), coef, token_mask=mask, seq_offsets=seqt, status=st)
    lg64 = lg.astype(np.float64)
    loss, c, P, n = ref_balance(lg64, idx, coef, keep, seq)
    assert np.array_equal(b["counts"].cpu().numpy(), c)
    assert np.array_equal(b["n_tokens"].cpu().numpy(), n)
    assert (np.abs(b["prob_mean"].cpu().numpy() - P) <= (1100 + E / 4) * U * P + 1e-38).all()
    assert abs(float(b["loss"]) - loss) <= (2200 + E) * U * abs(loss)
    d = moe.gate_topk_backward(cu(dev_lg), cu(idx), cu(dev_dw), renorm=renorm, balance=b,
                               d_loss=torch.full((1,), dl, device=DEV), token_mask=mask,
                               seq_offsets=seqt, status=st)
    ex, sc = ref_grad(lg64, idx, dw.astype(np.float64), renorm, keep, coef, seq, c, n, dl)
    got = d.cpu().numpy().astype(np.float64)
    assert int(st.item()) == 0
    assert (got[~keep] == 0).all()
    assert (np.abs(got - ex) <= (E + 64) * U * sc + 1e-38).all()
    # each part alone, and d_loss = 1 where it is not given
    only = moe.gate_topk_backward(cu(dev_lg), cu(idx), balance=b, token_mask=mask, seq_offsets=seqt)
    ex, sc = ref_grad(lg64, idx, None, renorm, keep, coef, seq, c, n, 1.0)
    assert (np.abs(only.cpu().numpy() - ex) <= (E + 64) * U * sc + 1e-38).all()
    only = moe.gate_topk_backward(cu(dev_lg), cu(idx), cu(dev_dw), renorm=renorm, token_mask=mask)
    ex, sc = ref_grad(lg64, idx, dw.astype(np.float64), renorm, keep, 0, seq, None, None, 0)
    assert (np.abs(only.cpu().numpy() - ex) <= (E + 64) * U * sc + 1e-38).all()


def test_no_tokens():
    lg, idx = torch.zeros(0, 8, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    b = moe.balance_loss(lg, idx, 1.0)
    assert float(b["loss"]) == 0 and not b["counts"].any() and not b["prob_mean"].any()
    assert moe.gate_topk_backward(lg, idx, balance=b).shape == (0, 8)


def test_uniform_router_has_loss_coef():
    T, E, k = 64, 16, 2
    idx = torch.arange(T * k, device=DEV, dtype=torch.int32).view(T, k) % E
    b = moe.balance_loss(torch.zeros(T, E, device=DEV), idx, 0.5)
    assert float(b["loss"]) == 0.5                 # every sum is of powers of two
    d = moe.gate_topk_backward(torch.zeros(T, E, device=DEV), idx, balance=b)
    assert not d.any()


def test_infinite_logits():
    """Experts switched off by -inf logits have no probability and no
    gradient; a row of nothing but -inf gives zeros."""
    rng, lg, idx, keep, seq = case(50, 24, 4, 1, 0.0, 9)
    lg[:, 3::5] = -np.inf
    lg[7] = -np.inf
    lg[8] = np.finfo(np.float32).min
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :4].astype(np.int32)
    dw = rng.standard_normal((50, 4)).astype(np.float32)
    b = moe.balance_loss(cu(lg), cu(idx), 1.0)
    loss, c, P, n = ref_balance(lg.astype(np.float64), idx, 1.0, keep, seq)
    assert (np.abs(b["prob_mean"].cpu().numpy() - P) <= 1100 * U * P).all()
    # row 8 alone (all logits equal) gives the switched-off experts anything
    assert (np.abs(P[0, 3::5] - 1.0 / (24 * 50)) <= 1e-15).all()
    for renorm in (True, False):
        d = moe.gate_topk_backward(cu(lg), cu(idx), cu(dw), renorm=renorm, balance=b)
        got = d.cpu().numpy()
        assert np.isfinite(got).all() and not got[7].any()
        assert not np.delete(got, 8, axis=0)[:, 3::5].any()
        rows = np.delete(np.arange(50), 7)
        ex, sc = ref_grad(lg[rows].astype(np.float64), idx[rows], dw[rows].astype(np.float64),
                          renorm, keep[rows], 1.0, [0, 49], c, n, 1.0)
        # tokens without row 7 see the same counts and n
        assert (np.abs(got[rows] - ex) <= 128 * U * sc).all()


def test_bad_ids_repeated_ids_and_bad_bounds():
    rng, lg, idx, keep, seq = case(40, 12, 4, 1, 0.0, 10)
    idx[3, 1] = 12
    idx[5, 0] = -1
    idx[6] = 2                                     # one expert four times
    dw = rng.standard_normal((40, 4)).astype(np.float32)
    st = moe.new_status(DEV)
    b = moe.balance_loss(cu(lg), cu(idx), 1.0, status=st)
    assert int(st.item()) == moe.DEV_BAD_EXPERT_ID
    loss, c, P, n = ref_balance(lg.astype(np.float64), idx, 1.0, keep, seq)
    assert np.array_equal(b["counts"].cpu().numpy(), c)
    for renorm in (True, False):
        st.zero_()
        d = moe.gate_topk_backward(cu(lg), cu(idx), cu(dw), renorm=renorm, balance=b, status=st)
        assert int(st.item()) == moe.DEV_BAD_EXPERT_ID
        ex, sc = ref_grad(lg.astype(np.float64), idx, dw.astype(np.float64), renorm, keep, 1.0, seq,
                          c, n, 1.0)
        assert (np.abs(d.cpu().numpy() - ex) <= 128 * U * sc).all()
    for bad in ([0, 41], [-1, 40], [20, 10]):
        st.zero_()
        moe.balance_loss(cu(lg), cu(idx), 1.0, seq_offsets=cu(np.array(bad, np.int32)), status=st)
        assert int(st.item()) & moe.DEV_BAD_OFFSETS
        st.zero_()
        moe.gate_topk_backward(cu(lg), cu(idx), cu(dw), balance=b, status=st,
                               seq_offsets=cu(np.array(bad, np.int32)))
        assert int(st.item()) & moe.DEV_BAD_OFFSETS


def test_gradient_against_differences():
    """Central differences of the loss and of a linear function of the weights
    in float64 (the assignments held), step 1e-5: error ~ 1e-10 of the scale."""
    rng, lg, idx, keep, seq = case(12, 10, 3, 2, 0.0, 12)
    seq = np.array([0, 5, 12], np.int32)
    dw = rng.standard_normal((12, 3))

    def f(z, renorm):
        loss = ref_balance(z, idx, 0.3, keep, seq)[0]
        w = np.take_along_axis(softmax(z), idx, 1)
        if renorm:
            w = w / w.sum(axis=1, keepdims=True)
        return loss + (w * dw).sum()
    b = moe.balance_loss(cu(lg), cu(idx), 0.3, seq_offsets=cu(seq))
    for renorm in (True, False):
        d = moe.gate_topk_backward(cu(lg), cu(idx), cu(dw.astype(np.float32)), renorm=renorm,
                                   balance=b, seq_offsets=cu(seq)).cpu().numpy()
        z = lg.astype(np.float64)
        for t, e in [(0, 0), (3, 9), (6, 4), (11, 2)] + [(t, idx[t, 1]) for t in range(12)]:
            zp, zm = z.copy(), z.copy()
            zp[t, e] += 1e-5
            zm[t, e] -= 1e-5
            num = (f(zp, renorm) - f(zm, renorm)) / 2e-5
            assert abs(num - d[t, e]) <= 1e-6


@pytest.mark.parametrize("E", [64, 200])
def test_rows_off_the_vector_alignment(E):
    """Logits that start 4 bytes behind a 16-byte boundary give the results of
    aligned ones, within the sums' rounding (their lanes hold other columns)."""
    rng, lg, idx, keep, seq = case(500, E, 6, 3, 0.1, 21)
    dw = cu(rng.standard_normal((500, 6)).astype(np.float32))
    buf = torch.zeros(500 * E + 1, device=DEV)
    off = buf[1:].view(500, E)
    off.copy_(cu(lg))
    assert off.data_ptr() % 16 == 4 and off.is_contiguous()
    res = []
    for z in (cu(lg), off):
        b = moe.balance_loss(z, cu(idx), 1.0, token_mask=cu(keep), seq_offsets=cu(seq))
        d = moe.gate_topk_backward(z, cu(idx), dw, balance=b, token_mask=cu(keep),
                                   seq_offsets=cu(seq))
        res.append((b, d.cpu().numpy().astype(np.float64)))
    loss, c, P, n = ref_balance(lg.astype(np.float64), idx, 1.0, keep, seq)
    ex, sc = ref_grad(lg.astype(np.float64), idx, dw.cpu().numpy().astype(np.float64), True, keep,
                      1.0, seq, c, n, 1.0)
    for b, d in res:
        assert np.array_equal(b["counts"].cpu().numpy(), c)
        assert (np.abs(b["prob_mean"].cpu().numpy() - P) <= (1100 + E / 4) * U * P).all()
        assert (np.abs(d - ex) <= (E + 64) * U * sc + 1e-38).all()


def test_long_sequences_and_offsets_past_32_bits():
    """T E beyond 2^31 elements: the last rows are reached (the values of a
    block of rows repeat, so the means are those of the block)."""
    E, block = 1024, 4096
    T = 2 ** 21 + 512 * 4
    rng = np.random.default_rng(3)
    lg = cu(rng.standard_normal((block, E)).astype(np.float32))
    big = lg.repeat(T // block + 1, 1)[:T].contiguous()
    idx = big.topk(2, dim=1).indices.to(torch.int32)
    st = moe.new_status(DEV)
    b = moe.balance_loss(big, idx, 1.0, status=st)
    ref = torch.softmax(big[T - T % block:].double(), 1).sum(0) if T % block else 0
    P = (torch.softmax(lg.double(), 1).sum(0) * (T // block) + ref) / T
    assert ((b["prob_mean"][0].double() - P).abs() <= 4000 * U * P).all()
    assert int(b["counts"].sum()) == 2 * T and int(st.item()) == 0
    d = moe.gate_topk_backward(big, idx, balance=b)
    few = moe.gate_topk_backward(big[:block].contiguous(), idx[:block].contiguous(), balance=b)
    assert torch.equal(d[T - T % block:] if T % block else d[-block:],
                       few[:T % block] if T % block else few)
    assert torch.equal(d[:block], few)


# ----------------------------------------------------------- finalize backward
@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (37, 2048, 8), (400, 264, 3), (310, 4104, 9),
                                   (5, 64, 32), (1000, 128, 2), (600, 1000, 12)])
@pytest.mark.parametrize("y32", [False, True])
@pytest.mark.parametrize("d32", [False, True])
def test_finalize_backward(T, H, k, y32, d32):
    g = torch.Generator().manual_seed(T + H)
    d = torch.randn((T, H), generator=g).to(torch.float32 if d32 else torch.bfloat16)
    y = torch.randn((T * k, H), generator=g).to(torch.float32 if y32 else torch.bfloat16)
    rows = torch.randperm(T * k, generator=g).to(torch.int32)
    w = torch.rand((T, k), generator=g)
    st = moe.new_status(DEV)
    dy, dw = moe.finalize_routing_backward(d.to(DEV), y.to(DEV), rows.to(DEV), w.to(DEV), status=st)
    assert int(st.item()) == 0 and dy.dtype == y.dtype
    r = rows.long().view(T, k)
    dd, yy = d.double(), y.double()
    ex = (dd[:, None, :] * yy[r]).sum(2)
    sc = (dd[:, None, :] * yy[r]).abs().sum(2)
    assert ((dw.cpu().double() - ex).abs() <= (H + 4) * U * sc).all()
    want = torch.empty((T * k, H), dtype=torch.float64)
    want[r.reshape(-1)] = (w.double()[:, :, None] * dd[:, None, :]).reshape(T * k, H)
    err = (dy.cpu().double() - want).abs()
    step = 2.0 ** -24 + (0.0 if y32 else 2.0 ** -8)
    assert (err <= step * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -140).all()


def test_finalize_backward_leaves_unnamed_rows_alone():
    T, H, k = 4, 64, 2
    d = torch.ones((T, H), dtype=torch.bfloat16, device=DEV)
    y = torch.ones((T * k, H), dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, -1, 2, 3, 4, 8, 6, 7], dtype=torch.int32, device=DEV)
    w = torch.full((T, k), 0.5, device=DEV)
    dy = torch.full((T * k, H), 9.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, k), 9.0, device=DEV)
    st = moe.new_status(DEV)
    moe._call("moe_finalize_routing_backward", moe._ptr(d), moe._ptr(y), moe._ptr(rows), moe._ptr(w),
              T, H, k, 0, moe._ptr(dy), moe._ptr(dw), moe._ptr(st), moe._stream(d.device))
    assert int(st.item()) == moe.DEV_BAD_OFFSETS
    assert (dy[[1, 5]] == 9.0).all() and (dy[[0, 2, 3, 4, 6, 7]] == 0.5).all()
    assert dw.view(-1).tolist() == [64.0, 0.0, 64.0, 64.0, 64.0, 0.0, 64.0, 64.0]


def test_repeats_streams_and_graphs():
    rng, lg, idx, keep, seq = case(3000, 64, 8, 5, 0.2, 14)
    lgc, idxc, m, sq = cu(lg), cu(idx), cu(keep), cu(seq)
    dw = cu(rng.standard_normal((3000, 8)).astype(np.float32))

    def step():
        b = moe.balance_loss(lgc, idxc, 0.1, token_mask=m, seq_offsets=sq)
        d = moe.gate_topk_backward(lgc, idxc, dw, balance=b, token_mask=m, seq_offsets=sq)
        return b["loss"], b["counts"], b["prob_mean"], d
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams * 3:
        with torch.cuda.stream(s):
            outs.append(step())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = step()
    for _ in range(2):
        for t in o:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want))


# --------------------------------------------------- a run of them together
@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_tuning_the_router_in_front_of_frozen_4_bit_experts(fmt):
    """Gate, balance loss, routing, 4-bit experts and the weighted sum, then
    back to the logits.  Against float64 on the routing, codes and rounded
    activations of the run itself; the weighted output and the gradient of a
    random linear function of it."""
    T, H, E, k, I = 200, 256, 8, 2, 128
    g = torch.Generator().manual_seed(5)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV)
    wg = (torch.randn((E, H), generator=g) * 0.05).to(DEV)
    w13 = moe.fp4_quantize((torch.randn((E, 2 * I, H), generator=g) * 0.05).bfloat16().to(DEV), fmt,
                           0 if fmt == "mx" else -5)
    w2 = moe.fp4_quantize((torch.randn((E, H, I), generator=g) * 0.05).bfloat16().to(DEV), fmt,
                          0 if fmt == "mx" else -5)
    d_out = torch.randn((T, H), generator=g).to(torch.bfloat16).to(DEV)
    st = moe.new_status(DEV)
    _, lg = moe.rmsnorm_gate(x, wg, rmsnorm=False)
    idx, w = moe.gate_topk(lg, k)
    bal = moe.balance_loss(lg, idx, 0.01, status=st)
    r = moe.init_routing(idx, x, E, with_rows=False, status=st)
    a = moe.fp4_quantize(x, fmt, row_idx=r["row_idx"], k=k, offsets=r["offsets"], status=st)
    act, y = moe.fp4_grouped_mlp(a, r["offsets"], w13, w2, y_f32=True, status=st)
    out = moe.finalize_routing(y, r["row_idx"], w, out_f32=True)
    d_y, d_w = moe.finalize_routing_backward(d_out, y, r["row_idx"], w, status=st)
    d_lg = moe.gate_topk_backward(lg, idx, d_w, balance=bal, status=st)
    assert int(st.item()) == 0
    assert torch.equal(bal["counts"][0], r["counts"])
    # products from the operands' exact values
    off = r["offsets"].tolist()
    av, actv = moe.fp4_dequantize(a, r["offsets"]).double(), moe.fp4_dequantize(act, r["offsets"]).double()
    ye = torch.zeros((T * k, H), dtype=torch.float64, device=DEV)
    ys = torch.zeros_like(ye)
    v2 = moe.fp4_dequantize(w2).double()
    for e in range(E):
        s = slice(off[e], off[e + 1])
        ye[s] = actv[s] @ v2[e].T
        ys[s] = actv[s].abs() @ v2[e].abs().T
    assert ((y.double() - ye).abs() <= (I + 8) * 2.0 ** -23 * ys).all()
    rows = r["row_idx"].long().view(T, k)
    z = lg.double().requires_grad_(True)
    p = torch.softmax(z, 1)
    sel = torch.gather(p, 1, idx.long())
    wt = sel / sel.sum(1, keepdim=True)
    o = (wt[:, :, None] * ye[rows]).sum(1)
    loss = 0.01 * E / (k * T) * (bal["counts"][0].double() * p.mean(0)).sum()
    ((o * d_out.double()).sum() + loss).backward()
    assert ((out.double() - o.detach()).abs() <= (I + 64) * 2.0 ** -23 * (wt.detach()[:, :, None] *
                                                                      ys[rows]).sum(1)).all()
    # d_w is off by (H + I + 12) fp32 steps of sum |d_out| ys per slot; the
    # renormalised weights' Jacobian rows sum to at most 1 in magnitude
    dws = (d_out.double().abs()[:, None, :] * ys[rows]).sum(2).max(1).values
    assert ((d_lg.double() - z.grad).abs() <= ((H + I + E + 80) * 2.0 ** -23 * dws)[:, None]).all()
