"""The block's newer operators at their limits: the most groups and sequences,
scratch memory that holds anything, several calls at once.  Tolerances as in the
operators' own tests, whose checks are used."""
import ctypes

import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe
from . import test_gpu_fp4_weight as w4
from . import test_gpu_mlp_train as mlp
from . import test_gpu_norm_residual as nr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64 = torch.float64


def spread(G, active, most, seed):
    """Rows of G groups, `active` of them with up to `most`."""
    g = torch.Generator().manual_seed(seed)
    c = torch.zeros(G, dtype=torch.int64)
    c[torch.randperm(G, generator=g)[:active]] = torch.randint(1, most + 1, (active,), generator=g)
    return c.tolist()


@pytest.mark.parametrize("G,active,most", [(1024, 300, 3), (1024, 1024, 1), (300, 280, 200), (480, 5, 600),
                                           (481, 400, 9)])
def test_many_groups_trained(G, active, most):
    counts = spread(G, active, most, G + most)
    x, off, w13, w2, d_y = mlp.make(counts, 128, 128, G)
    st = moe.new_status(DEV)
    h, y = moe.grouped_mlp_train(x, off, w13, w2, status=st)
    assert torch.equal(y, moe.grouped_mlp(x, off, w13, w2)[1])
    got = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, status=st)
    f32 = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=True, status=st)
    assert int(st.item()) == 0
    some = [g for g in range(G) if counts[g]][:: max(1, active // 12)] + [g for g in range(G) if not counts[g]][:3]
    o = off.tolist()
    for g in some:
        a, b = o[g], o[g + 1]
        one = torch.tensor([0, b - a], dtype=torch.int32, device=DEV)
        mlp.check_forward(x[a:b], one, w13[g:g + 1], w2[g:g + 1], h[a:b], y[a:b])
        for res, f in ((got, False), (f32, True)):
            mlp.check_backward(x[a:b], one, w13[g:g + 1], w2[g:g + 1], h[a:b], d_y[a:b],
                               (res[0][a:b], res[1][g:g + 1], res[2][g:g + 1]), w_f32=f)


@pytest.mark.parametrize("counts,H,I", [([300, 20, 513], 256, 384), ([8300], 128, 256), ([40, 3], 384, 128)])
def test_both_gradient_tiles(counts, H, I):
    """Sizes on both sides of the rule that picks the gradients' tiles, with
    sizes of 128 modulo either."""
    x, off, w13, w2, d_y = mlp.make(counts, H, I, H)
    h, _ = moe.grouped_mlp_train(x, off, w13, w2)
    for f in (False, True):
        mlp.check_backward(x, off, w13, w2, h, d_y,
                           moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=f), w_f32=f)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_many_groups_of_weights(fmt):
    counts = spread(1024, 200, 11, 3)
    x, off = w4.rows_of(counts, 256, 4)
    m, w = w4.weights(1024, 128, 256, fmt, 5)
    w4.check_matmul(x, off, w, moe.fp4_weight_matmul(x, off, m, out_f32=True), True)


def test_nonfinite_rows_in_the_gate():
    """SwiGLU of rows with infinities: what the formula gives for the sums."""
    x, off = w4.rows_of([3, 9], 256, 6)
    x = (x.float() / 64).to(torch.bfloat16)
    m, w = w4.weights(2, 256, 256, "nv", 7, -3)
    x[1, 5], x[7, 3] = float("inf"), float("nan")
    act = moe.fp4_weight_swiglu(x, off, m, out_f32=True)
    plain = moe.fp4_weight_matmul(x, off, m, out_f32=True)
    for r in (1, 7):
        g, u = plain[r, :128].to(F64), plain[r, 128:].to(F64)
        want = g / (1 + torch.exp(-g)) * u
        assert torch.equal(torch.isnan(act[r]), torch.isnan(want))
        assert torch.equal(act[r][torch.isinf(want)].to(F64), want[torch.isinf(want)])
    keep = [r for r in range(12) if r not in (1, 7)]
    o2 = torch.tensor([0, 2, 10], dtype=torch.int32, device=DEV)
    w4.check_swiglu(x[keep], o2, w, act[keep], True)


def test_many_sequences():
    T, H, S = 3000, 64, 65536
    cuts = torch.randint(0, T + 1, (S - 1,), generator=torch.Generator().manual_seed(8)).sort().values.tolist()
    seq = [0] + cuts + [T]
    d = nr.make(T, H, seq, 9)
    kw = dict(gamma_post=d["gp"], gate=d["gate"], scale=0.7, gamma_next=d["gn"], seq_offsets=d["seq"])
    f = moe.norm_residual(d["x"], d["y"], eps=nr.EPS, **kw)
    nr.check_forward(d, seq, f, 0.7, True, True)
    g = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, **kw)
    lens = torch.tensor(seq[1:]) - torch.tensor(seq[:-1])
    assert not g["d_gate"][(lens == 0).to(DEV)].any()
    # the same rows under one gate row each: sums over all sequences agree
    rep = torch.repeat_interleave(torch.arange(S), lens).to(DEV)
    dx, yh = g["d_x"].to(F64), d["y"].to(F64) * f["rstd_post"].to(F64)[:, None]
    want = torch.zeros(S, H, dtype=F64, device=DEV).index_add_(0, rep, 0.7 * dx * yh * d["gp"].to(F64))
    err = (g["d_gate"].to(F64) - want).abs()
    # d_x is bf16 here: b of each term
    mag = torch.zeros(S, H, dtype=F64, device=DEV).index_add_(0, rep, (0.7 * dx * yh * d["gp"].to(F64)).abs())
    assert (err <= 1.1 * nr.B * mag + 1e-30).all()


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def test_scratch_memory_may_hold_anything():
    L, s = moe.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    x, off, w13, w2, d_y = mlp.make([130, 0, 61], 256, 256, 10)
    h, _ = moe.grouped_mlp_train(x, off, w13, w2)
    want = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
    xq, offq = w4.rows_of([9, 1, 0, 3], 2048, 11)
    m, _ = w4.weights(4, 256, 2048, "mx", 12)
    wantq = moe.fp4_weight_matmul(xq, offq, m)
    d = nr.make(300, 512, [0, 100, 300], 13)
    kw = dict(gamma_post=d["gp"], gate=d["gate"], gamma_next=d["gn"], seq_offsets=d["seq"])
    f = moe.norm_residual(d["x"], d["y"], **kw)
    wantn = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, **kw)
    for fill in (0xFF, 0x7F, 0x01):
        ws = torch.full((moe.grouped_mlp_backward_workspace_size(191, 256),), fill, dtype=torch.uint8, device=DEV)
        got = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        n = moe.fp4_weight_workspace_size(13, 2048, 256, 4)
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(wantq)
        assert L.moe_fp4_weight_matmul(_ptr(xq), _ptr(offq), 4, moe._fp4_arg(m, "w", 0, xq.device), 13, 2048, 256, 0,
                                       _ptr(out), _ptr(ws), n, None, s) == 0
        assert torch.equal(out, wantq)
        n = moe.norm_residual_backward_workspace_size(300, 512, 2)
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        o = {k: torch.empty_like(v) for k, v in wantn.items()}
        assert L.moe_norm_residual_backward(
            _ptr(d["d_r"]), _ptr(d["d_xn"]), _ptr(d["y"]), _ptr(f["r"]), _ptr(f["rstd_post"]), _ptr(f["rstd_next"]),
            _ptr(d["gp"]), _ptr(d["gate"]), _ptr(d["seq"]), 2, _ptr(d["gn"]), 300, 512, 1.0, moe.POST_NORM,
            _ptr(o["d_x"]), _ptr(o["d_y"]), _ptr(o["d_gamma_post"]), _ptr(o["d_gate"]), _ptr(o["d_gamma_next"]),
            _ptr(ws), n, None, s) == 0
        assert all(torch.equal(o[k], wantn[k]) for k in o)


def test_several_streams_at_once():
    """The operators interleaved on four streams, each with its own memory."""
    x, off, w13, w2, d_y = mlp.make([300, 77, 0, 140], 512, 256, 14)
    xq, offq = w4.rows_of([5, 12], 1024, 15)
    m, _ = w4.weights(2, 512, 1024, "nv", 16)
    d = nr.make(600, 1024, [0, 250, 600], 17)
    kw = dict(gamma_post=d["gp"], gate=d["gate"], gamma_next=d["gn"], seq_offsets=d["seq"])

    def step():
        h, y = moe.grouped_mlp_train(x, off, w13, w2)
        f = moe.norm_residual(d["x"], d["y"], **kw)
        a = moe.fp4_weight_swiglu(xq, offq, m)
        g = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
        b = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, **kw)
        return [h, y, a, *g, *f.values(), *b.values()]

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_two_blocks_step():
    """Norm, routing, experts, weighted sum, norm: a step through the residual
    stream with every gradient, captured into a graph, against autograd in 64
    bits on the same expert choice."""
    T, H, I, E, k, S = 160, 256, 128, 8, 2, 2
    g = torch.Generator().manual_seed(18)
    rnd = lambda *s: torch.randn(*s, generator=g)                          # noqa: E731
    bf = lambda t: t.to(torch.bfloat16).to(DEV)                            # noqa: E731
    x, y0, d_r, d_xn = rnd(T, H).to(DEV), bf(rnd(T, H)), (rnd(T, H) * 0.1).to(DEV), bf(rnd(T, H) * 0.1)
    gam = [bf(1 + 0.1 * rnd(H)) for _ in range(4)]
    gate = [bf(rnd(S, H)) for _ in range(2)]
    seq = torch.tensor([0, 70, T], dtype=torch.int32, device=DEV)
    wg = (rnd(E, H) * 0.1).to(DEV)
    w13, w2 = bf(rnd(E, 2 * I, H) / H ** 0.5), bf(rnd(E, H, I) / I ** 0.5)
    n0 = dict(gamma_post=gam[0], gate=gate[0], scale=0.5, gamma_next=gam[1], seq_offsets=seq)
    n1 = dict(gamma_post=gam[2], gate=gate[1], scale=0.5, gamma_next=gam[3], seq_offsets=seq)

    def step():
        a = moe.norm_residual(x, y0, **n0)
        logits = moe.gate_tensor(a["xn"], wg)
        idx, w = moe.gate_topk(logits, k)
        r = moe.init_routing(idx, a["xn"], E)
        h, y = moe.grouped_mlp_train(r["expanded_x"], r["offsets"], w13, w2)
        out = moe.finalize_routing(y, r["row_idx"], w)
        b = moe.norm_residual(a["r"], out, **n1)
        db = moe.norm_residual_backward(d_r, d_xn, out, b, **n1)
        d_y, d_w = moe.finalize_routing_backward(db["d_y"], y, r["row_idx"], w)
        d_ex, d_w13, d_w2 = moe.grouped_mlp_backward(d_y, r["expanded_x"], r["offsets"], h, w13, w2)
        d_lg = moe.gate_topk_backward(logits, idx, d_w)
        # the rows' gradients back to the tokens (and what the gate adds)
        d_n = moe.finalize_routing(d_ex, r["row_idx"], torch.ones_like(w), out_f32=True) + d_lg @ wg
        da = moe.norm_residual_backward(db["d_x"], d_n.to(torch.bfloat16), y0, a, **n0)
        return dict(idx=idx, r=b["r"], xn=b["xn"], d_x=da["d_x"], d_y0=da["d_y"], d_g0=da["d_gamma_post"],
                    d_g1=da["d_gamma_next"], d_g2=db["d_gamma_post"], d_g3=db["d_gamma_next"],
                    d_gate0=da["d_gate"], d_gate1=db["d_gate"], d_w13=d_w13, d_w2=d_w2)

    got = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    graph.replay()
    for key in got:
        assert torch.equal(got[key], cap[key]), key

    p = {n: t.to(F64).requires_grad_() for n, t in
         dict(x=x, y0=y0, g0=gam[0], g1=gam[1], g2=gam[2], g3=gam[3], gate0=gate[0], gate1=gate[1], w13=w13,
              w2=w2).items()}
    sid = torch.cat((torch.zeros(70), torch.ones(T - 70))).long().to(DEV)

    def norm(v, gm):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * gm

    r0 = p["x"] + 0.5 * p["gate0"][sid] * norm(p["y0"], p["g0"])
    xn = norm(r0, p["g1"])
    lg = xn @ wg.to(F64).T
    idx = got["idx"].long()
    sel = torch.gather(torch.softmax(lg, 1), 1, idx)
    sel = sel / sel.sum(1, keepdim=True)
    out = torch.zeros(T, H, dtype=F64, device=DEV)
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        v = xn[t] @ p["w13"][e].T
        out = out.index_add(0, t, (torch.nn.functional.silu(v[:, :I]) * v[:, I:]) @ p["w2"][e].T * sel[t, j][:, None])
    r1 = r0 + 0.5 * p["gate1"][sid] * norm(out, p["g2"])
    xn1 = norm(r1, p["g3"])
    loss = (d_r.to(F64) * r1).sum() + (d_xn.to(F64) * xn1).sum()
    grads = dict(zip(p, torch.autograd.grad(loss, list(p.values()))))
    want = dict(r=r1.detach(), xn=xn1.detach(), **{"d_" + n: v for n, v in grads.items()})
    # bf16 roundings on the way to a gradient: xn, h, act, y, out, d_out, d_y, d_h, d_ex,
    # d_n and the result's own, each b / sqrt(3) at most in the mean square
    for key, v in want.items():
        err = float((got[key].to(F64) - v).norm() / v.norm())
        assert err <= 11 ** 0.5 * nr.B / 3 ** 0.5, (key, err)


@pytest.mark.parametrize("H,I", [(256, 256), (512, 384), (128, 128)])
def test_ragged_groups_again(H, I):
    """Groups whose last rows are stored row by row (31 and 127 mod 128 of them):
    pass after pass has the same bits."""
    x, off, w13, w2, d_y = mlp.make([127, 255, 31, 191] * 20, H, I, I)
    h, y = moe.grouped_mlp_train(x, off, w13, w2)
    want = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
    mlp.check_backward(x, off, w13, w2, h, d_y, want)
    for _ in range(150):
        h1, y1 = moe.grouped_mlp_train(x, off, w13, w2)
        got = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
        assert torch.equal(h, h1) and torch.equal(y, y1)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_in_front_of_the_first_group():
    """Offsets may start behind row 0; what the rows in front hold enters nothing."""
    x, off, w13, w2, d_y = mlp.make([37, 0, 300, 5], 256, 384, 4)
    h, y = moe.grouped_mlp_train(x, off, w13, w2)
    want = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
    nan = torch.full((21, 768), float("nan"), dtype=torch.bfloat16, device=DEV)
    front = lambda t: torch.cat((nan[:, :t.shape[1]], t))                  # noqa: E731
    off2 = off + 21
    h2, y2 = moe.grouped_mlp_train(front(x), off2, w13, w2)
    got = moe.grouped_mlp_backward(front(d_y), front(x), off2, front(h), w13, w2)
    assert torch.equal(h2[21:], h) and torch.equal(y2[21:], y) and torch.equal(got[0][21:], want[0])
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
