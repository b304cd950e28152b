"""The expert FFN's training passes against the formulas in float64.

Rounding model (u = 2^-24 an fp32 half step, b = 2^-8 a bf16 one): a product of
K terms accumulated in fp32 is off by at most 2 K u sum|terms| (the tensor cores
may truncate); sigmoid by the hardware exponential and reciprocal is within
2^-20 relative; every bf16 result adds b of itself.  The bounds propagate these
through the next product as sums of absolute values.  As those grow with the
number of terms where errors only grow with its root, the relative 2-norm is
held too: a bf16 rounding's errors are at most b / sqrt(3) in the mean square
(uniform in the last place), 2.3e-3; h and d_x, d_w13 (rounded themselves, their
operand once before) stay under 2 b / sqrt(3) = 4.6e-3, y (act rounded, y
rounded) likewise.
"""
import ctypes

import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, B = 2.0 ** -24, 2.0 ** -8
NORM = 4.6e-3
F64 = torch.float64


def make(counts, H, I, seed, tail=0, scale=1.0):
    """Rows of each group, `tail` rows behind the last one."""
    g = torch.Generator().manual_seed(seed)
    n = sum(counts) + tail
    rnd = lambda *s: torch.randn(*s, generator=g)                       # noqa: E731
    x = (rnd(n, H) * scale).to(torch.bfloat16)
    w13 = (rnd(len(counts), 2 * I, H) / H ** 0.5).to(torch.bfloat16)
    w2 = (rnd(len(counts), H, I) / I ** 0.5).to(torch.bfloat16)
    d_y = (rnd(n, H) * 0.1).to(torch.bfloat16)
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(counts), 0)
    return [t.to(DEV) for t in (x, off, w13, w2, d_y)]


def near(got, want, tol, name, norm=NORM):
    got = got.to(F64)
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    bad = err > tol
    assert not bad.any(), (name, float((err / tol.clamp(min=1e-300)).max()), int(bad.sum()))
    if norm is not None and float(want.norm()) > 0:
        assert float((got - want).norm() / want.norm()) <= norm, name


def check_forward(x, off, w13, w2, h, y):
    I, H = w2.shape[2], w2.shape[1]
    o = off.tolist()
    for g in range(len(o) - 1):
        a, b = o[g], o[g + 1]
        if a == b:
            continue
        X, W, V = x[a:b].to(F64), w13[g].to(F64), w2[g].to(F64)
        ref = X @ W.T
        e = 2 * H * U * (X.abs() @ W.abs().T)
        near(h[a:b], ref, B * ref.abs() + e, "h")
        gate, up = ref[:, :I], ref[:, I:]
        s = torch.sigmoid(gate)
        act = gate * s * up
        # |SiLU'| <= 1.1
        ea = B * act.abs() + 2.0 ** -19 * act.abs() + 1.1 * e[:, :I] * up.abs() + \
            (gate * s).abs() * e[:, I:] + e[:, :I] * e[:, I:]
        yr = act @ V.T
        near(y[a:b], yr, B * yr.abs() + ea @ V.abs().T + 2 * I * U * (act.abs() @ V.abs().T), "y")


def reference_backward(x, off, w13, w2, h, d_y):
    """Per group: (rows, the gradients and their tolerances without the
    results' own rounding)."""
    I, H = w2.shape[2], w2.shape[1]
    o = off.tolist()
    for g in range(len(o) - 1):
        a, b = o[g], o[g + 1]
        X, W, V, D = x[a:b].to(F64), w13[g].to(F64), w2[g].to(F64), d_y[a:b].to(F64)
        gate, up = h[a:b, :I].to(F64), h[a:b, I:].to(F64)
        s = torch.sigmoid(gate)
        gs = gate * s
        d = D @ V
        ed = 2 * H * U * (D.abs() @ V.abs()) + 2.0 ** -19 * d.abs()
        dh = torch.cat((d * up * (s + gs * (1 - s)), d * gs), 1)
        eh = B * dh.abs() + (1 + B) * torch.cat((ed * up.abs() * (s + gs.abs() * (1 - s)),
                                                 ed * gs.abs()), 1)
        # 1 / (1 + e^-gate) with a sum from 2^126 on (gate < -87.3) is taken as zero:
        # s is off by s < 2^-126 then, gs by |gate| 2^-126
        lost = torch.where(gate < -87.3, 2.0 ** -126, 0.0)
        eh = eh + lost.repeat(1, 2) * torch.cat((d.abs() * up.abs() * (1 + gate.abs()),
                                                 d.abs() * gate.abs()), 1)
        act = gs * up
        ea = (B + 2.0 ** -19) * act.abs() + lost * gate.abs() * up.abs()
        dx = dh @ W
        ex = eh @ W.abs() + 4 * I * U * (dh.abs() @ W.abs())
        dw, ew = dh.T @ X, eh.T @ X.abs() + 2 * (b - a) * U * (dh.abs().T @ X.abs())
        dv, ev = D.T @ act, D.abs().T @ ea + 2 * (b - a) * U * (D.abs().T @ act.abs())
        yield g, a, b, (dx, ex), (dw, ew), (dv, ev)


def check_backward(x, off, w13, w2, h, d_y, got, w_f32=False, base=(0.0, 0.0)):
    rb = 0.0 if w_f32 else B
    for g, a, b, (dx, ex), (dw, ew), (dv, ev) in reference_backward(x, off, w13, w2, h, d_y):
        if got[0] is not None and b > a:
            near(got[0][a:b], dx, B * dx.abs() + ex, "d_x")
        for k, (r, e, bs) in enumerate(((dw, ew, base[0]), (dv, ev, base[1]))):
            t = got[1 + k]
            if t is None:
                continue
            if not isinstance(bs, float):
                r, e = r + bs[g], e + U * (r + bs[g]).abs()
            elif b == a:
                assert not t[g].any(), "an idle expert's gradient"
                continue
            near(t[g], r, rb * r.abs() + e + 1e-30, ("d_w13", "d_w2")[k])


SHAPES = [
    ([1], 128, 128), ([5], 256, 128), ([130], 128, 256), ([257], 384, 384),
    ([0, 3, 0, 1], 128, 128), ([64, 16, 15, 17], 256, 256), ([300, 0, 128, 129, 1], 256, 384),
    ([127, 128, 255, 256], 512, 256), ([1000, 400], 640, 128), ([16, 512, 33], 128, 640),
    ([2] * 40 + [0] * 24, 256, 256), ([200] * 7, 256, 128), ([700, 1, 0, 900], 1024, 512),
]


@pytest.mark.parametrize("counts,H,I", SHAPES)
def test_forward_and_backward(counts, H, I):
    x, off, w13, w2, d_y = make(counts, H, I, sum(counts) + H)
    st = moe.new_status(DEV)
    h, y = moe.grouped_mlp_train(x, off, w13, w2, status=st)
    check_forward(x, off, w13, w2, h, y)
    _, plain = moe.grouped_mlp(x, off, w13, w2)
    assert torch.equal(y, plain)
    got = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, status=st)
    check_backward(x, off, w13, w2, h, d_y, got)
    f32 = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=True, status=st)
    check_backward(x, off, w13, w2, h, d_y, f32, w_f32=True)
    assert torch.equal(f32[0].view(torch.int16), got[0].view(torch.int16))
    assert int(st.item()) == 0


def test_other_rows_do_not_enter():
    """Infinities and NaN behind the last group and in another group's rows."""
    counts, H, I = [130, 37, 0, 61], 256, 256
    x, off, w13, w2, d_y = make(counts, H, I, 5, tail=90)
    n = sum(counts)
    h, _ = moe.grouped_mlp_train(x, off, w13, w2)
    want = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
    check_backward(x, off, w13, w2, h, d_y, want)
    for t in (x, d_y, h):
        t[n:] = float("nan")
        t[130:167] = float("inf")
    got = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
    for g in (0, 2, 3):
        a, b = int(off[g]), int(off[g + 1])
        assert torch.equal(got[0][a:b], want[0][a:b])
        assert torch.equal(got[1][g], want[1][g]) and torch.equal(got[2][g], want[2][g])


def test_rows_behind_the_last_group_are_left():
    counts, H, I = [130, 0, 37], 256, 128
    x, off, w13, w2, d_y = make(counts, H, I, 6, tail=50)
    n, N = sum(counts), x.shape[0]
    L, p = moe.lib(), lambda t: ctypes.c_void_p(t.data_ptr())             # noqa: E731
    h = torch.full((N, 2 * I), 7.0, dtype=torch.bfloat16, device=DEV)
    act, y, d_x = (torch.full((N, c), 7.0, dtype=torch.bfloat16, device=DEV) for c in (I, H, H))
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.moe_grouped_mlp_train(p(x), p(off), 3, p(w13), p(w2), N, H, I, p(h), p(act), p(y),
                                   None, s) == 0
    ws = torch.empty(moe.grouped_mlp_backward_workspace_size(N, I), dtype=torch.uint8,
                     device=DEV)
    assert L.moe_grouped_mlp_backward(p(d_y), p(x), p(off), 3, p(h), p(w13), p(w2), N, H, I, 0,
                                      p(d_x), None, None, p(ws), ws.numel(), None, s) == 0
    for t in (h, act, y, d_x):
        assert (t[n:] == 7.0).all() and not (t[:n] == 7.0).all()


def test_accumulate_adds_in_fp32():
    counts, H, I = [140, 0, 33], 128, 256
    x, off, w13, w2, d_y = make(counts, H, I, 7)
    h, _ = moe.grouped_mlp_train(x, off, w13, w2)
    b13, b2 = torch.randn((3, 2 * I, H), device=DEV), torch.randn((3, H, I), device=DEV)
    a13, a2 = b13.clone(), b2.clone()
    got = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=True, d_w13=a13, d_w2=a2,
                                   accumulate=True)
    assert got[1] is a13 and got[2] is a2
    plain = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=True)
    assert torch.equal(a13, b13 + plain[1]) and torch.equal(a2, b2 + plain[2])
    check_backward(x, off, w13, w2, h, d_y, got, w_f32=True, base=(b13.to(F64), b2.to(F64)))


@pytest.mark.parametrize("need", [("x",), ("w13",), ("w2",), ("x", "w2"), ()])
def test_parts(need):
    x, off, w13, w2, d_y = make([70, 0, 200], 256, 256, 8)
    h, _ = moe.grouped_mlp_train(x, off, w13, w2)
    full = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
    part = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, need=need)
    for name, f, t in zip(("x", "w13", "w2"), full, part):
        assert (t is None) == (name not in need)
        assert t is None or torch.equal(t, f)


def test_no_rows():
    x, off, w13, w2, d_y = make([0, 0], 128, 128, 9)
    h, y = moe.grouped_mlp_train(x, off, w13, w2)
    assert h.shape == (0, 256) and y.shape == (0, 128)
    d = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2)
    assert d[0].shape == (0, 128) and not d[1].any() and not d[2].any()
    # rows, but none in a group
    x, _, w13, w2, d_y = make([0, 0], 128, 128, 9, tail=40)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    h, y = moe.grouped_mlp_train(x, off, w13, w2)
    d = moe.grouped_mlp_backward(d_y, x, off, h.zero_(), w13, w2)
    assert not d[1].any() and not d[2].any()


@pytest.mark.parametrize("off", [[0, 5, 3], [-1, 4, 8], [0, 4, 9]])
def test_bad_offsets_write_nothing(off):
    x, _, w13, w2, d_y = make([4, 4], 128, 128, 10)
    off = torch.tensor(off, dtype=torch.int32, device=DEV)
    h = torch.zeros((8, 256), dtype=torch.bfloat16, device=DEV)
    st = moe.new_status(DEV)
    moe.grouped_mlp_train(x, off, w13, w2, status=st)
    assert int(st.item()) == moe.DEV_BAD_OFFSETS
    st.zero_()
    d13 = torch.full((2, 256, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    d2 = torch.full((2, 128, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, d_w13=d13, d_w2=d2, status=st)
    assert int(st.item()) == moe.DEV_BAD_OFFSETS
    assert (d13 == 3.0).all() and (d2 == 3.0).all()


def test_extreme_gates():
    """Gates far out on both sides: SiLU's derivative is 0 and 1 there."""
    x, off, w13, w2, d_y = make([40], 128, 128, 11)
    h = torch.randn((40, 256), device=DEV).to(torch.bfloat16)
    h[:, :128] = torch.linspace(-3e4, 3e4, 128, device=DEV).to(torch.bfloat16)
    h[3, :128] = -88.5
    h[4, :128] = 0.0
    h[5, :128] = 3e38
    h[6, :128] = -3e38
    d = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=True)
    for t in d[:2]:
        assert torch.isfinite(t).all()
    keep = [i for i in range(40) if i not in (5, 6)]
    xs, hs, ds = x[keep], h[keep], d_y[keep]
    off = torch.tensor([0, 38], dtype=torch.int32, device=DEV)
    check_backward(xs, off, w13, w2, hs, ds,
                   moe.grouped_mlp_backward(ds, xs, off, hs, w13, w2, w_f32=True), w_f32=True)


def test_against_differences():
    """Directional differences of sum(d_y * y) in float64.  The kernels take
    the gradient at the bf16 h they kept and round once more on the way: per
    gradient the relative 2-norm is within three roundings, 3 b / sqrt(3), of the
    true one, and so is its product with any direction, relative to both norms."""
    x, off, w13, w2, d_y = make([50, 0, 90], 256, 128, 12)
    h, _ = moe.grouped_mlp_train(x, off, w13, w2)
    got = moe.grouped_mlp_backward(d_y, x, off, h, w13, w2, w_f32=True)

    def loss(x, w13, w2):
        t = 0.0
        for g, a, b in ((0, 0, 50), (2, 50, 140)):
            v = x[a:b] @ w13[g].T
            t = t + ((torch.nn.functional.silu(v[:, :128]) * v[:, 128:]) @ w2[g].T *
                     d_y[a:b].to(F64)).sum()
        return float(t)

    p = [t.to(F64) for t in (x, w13, w2)]
    for k in range(3):
        v = got[k].to(F64)
        v = v / v.norm() * p[k].norm()
        up, dn = list(p), list(p)
        up[k], dn[k] = p[k] + 1e-5 * v, p[k] - 1e-5 * v
        diff = (loss(*up) - loss(*dn)) / 2e-5
        assert abs(float((got[k].to(F64) * v).sum()) - diff) <= \
            3 * B / 3 ** 0.5 * float(got[k].to(F64).norm() * v.norm())


def test_captured_replayed_and_on_another_stream():
    x, off, w13, w2, d_y = make([300, 0, 77, 129], 256, 256, 13)
    h0, y0 = moe.grouped_mlp_train(x, off, w13, w2)
    want = moe.grouped_mlp_backward(d_y, x, off, h0, w13, w2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h1, y1 = moe.grouped_mlp_train(x, off, w13, w2)
        other = moe.grouped_mlp_backward(d_y, x, off, h1, w13, w2)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y0, y1) and all(torch.equal(a, b) for a, b in zip(want, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h2, y2 = moe.grouped_mlp_train(x, off, w13, w2)
        cap = moe.grouped_mlp_backward(d_y, x, off, h2, w13, w2)
    for t in (h2, y2, *cap):
        t.zero_()
    g.replay()
    assert torch.equal(y0, y2) and all(torch.equal(a, b) for a, b in zip(want, cap))
    # other rows and other groups under the same graph
    x.copy_(x.roll(7, 0))
    off.copy_(torch.tensor([0, 10, 300, 300, 506], dtype=torch.int32))
    h3, y3 = moe.grouped_mlp_train(x, off, w13, w2)
    again = moe.grouped_mlp_backward(d_y, x, off, h3, w13, w2)
    g.replay()
    assert torch.equal(y3, y2) and all(torch.equal(a, b) for a, b in zip(again, cap))


def test_training_step_of_the_block():
    """The operators of a block's step together: routing, the FFN, the weighted
    sum, and every gradient back to the tokens and the gate."""
    T, H, I, E, k = 200, 256, 128, 8, 2
    g = torch.Generator().manual_seed(14)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    wg = (torch.randn(E, H, generator=g) * 0.1).to(DEV)
    w13 = (torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).to(torch.bfloat16).to(DEV)
    w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).to(torch.bfloat16).to(DEV)
    d_out = (torch.randn(T, H, generator=g) * 0.1).to(torch.bfloat16).to(DEV)
    logits = moe.gate_tensor(x, wg)
    idx, w = moe.gate_topk(logits, k)
    r = moe.init_routing(idx, x, E)
    h, y = moe.grouped_mlp_train(r["expanded_x"], r["offsets"], w13, w2)
    out = moe.finalize_routing(y, r["row_idx"], w)
    d_y, d_w = moe.finalize_routing_backward(d_out, y, r["row_idx"], w)
    d_ex, d_w13, d_w2 = moe.grouped_mlp_backward(d_y, r["expanded_x"], r["offsets"], h, w13, w2)
    d_x = moe.finalize_routing(d_ex, r["row_idx"], torch.ones_like(w), out_f32=True)
    d_lg = moe.gate_topk_backward(logits, idx, d_w)
    # autograd in 64 bits on the same expert choice
    p = [t.to(F64).requires_grad_() for t in (x, w13, w2, logits)]
    sel = torch.gather(torch.softmax(p[3], 1), 1, idx.long())
    sel = sel / sel.sum(1, keepdim=True)
    ref = torch.zeros(T, H, dtype=F64, device=DEV)
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        v = p[0][t] @ p[1][e].T
        f = (torch.nn.functional.silu(v[:, :I]) * v[:, I:]) @ p[2][e].T
        ref = ref.index_add(0, t, f * sel[t, j][:, None])
    grads = torch.autograd.grad((ref * d_out.to(F64)).sum(), p)
    # roundings on the way: y, d_y, d_h, act, h and the results' own
    for got, want, name in ((out, ref.detach(), "out"), (d_x, grads[0], "d_x"),
                            (d_w13, grads[1], "d_w13"), (d_w2, grads[2], "d_w2"),
                            (d_lg, grads[3], "d_logits")):
        assert float((got.to(F64) - want).norm() / want.norm()) <= 6 ** 0.5 * B, name
