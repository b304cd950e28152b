"""norm_residual and its backward pass against float64.

Rounding model (u = 2^-24, b = 2^-8): a sum of H terms in pieces is off by at
most (H / 256 + 24) 2 u of sum|terms| (a lane adds up to H / 256 + 8 of them in a
row, then 5 steps in the warp, 8 across); k = 1 / sqrt(.) by 8 u relative beyond
half of its sum's; elementwise products a few u each, counted as 16 u; results in
bf16 b of themselves.  Column sums over T rows: (T / 300 + 320) 2 u of
sum|terms| besides the terms' own errors (a team adds its rows in order, then
at most 320 teams' sums in a row).
"""
import pytest
import torch

import moe_expert_routing_fp32_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, B = 2.0 ** -24, 2.0 ** -8
F64 = torch.float64
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def make(T, H, seq, seed, xt=BF, yt=BF, gated=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)                        # noqa: E731
    S = len(seq) - 1 if seq else 1
    d = dict(x=(rnd(T, H) * 2).to(xt), y=rnd(T, H).to(yt), gp=(1 + 0.2 * rnd(H)).to(BF),
             gn=(1 + 0.2 * rnd(H)).to(BF), gate=rnd(S, H).to(BF) if gated else None,
             seq=torch.tensor(seq, dtype=torch.int32) if seq else None,
             d_r=(rnd(T, H) * 0.1).to(xt), d_xn=(rnd(T, H) * 0.1).to(BF))
    return {k: v.to(DEV) if v is not None else None for k, v in d.items()}


def near(got, want, tol, name):
    assert torch.isfinite(got).all(), name
    err = (got.to(F64) - want).abs()
    assert (err <= tol + 1e-37).all(), (name, float((err / (tol + 1e-37)).max()))


def rows_in(seq, T):
    m = torch.ones(T, dtype=torch.bool, device=DEV)
    if seq:
        m[:seq[0]] = False
        m[seq[-1]:] = False
    return m


def gate_of(d, seq, T):
    if d["gate"] is None:
        return 1.0
    s = torch.tensor(seq if seq else [0, T], device=DEV)
    sid = torch.searchsorted(s[1:].contiguous(), torch.arange(T, device=DEV), right=True)
    return d["gate"].to(F64)[sid.clamp(max=len(s) - 2)]


def rel_k(H):
    """Relative error of 1 / sqrt(mean + eps)."""
    return (H / 256 + 24) * U + 8 * U


def check_forward(d, seq, f, scale, post, nxt):
    T, H = d["x"].shape
    m = rows_in(seq, T)
    x, y = d["x"].to(F64), d["y"].to(F64)
    gp = d["gp"].to(F64) if post else 1.0
    k = 1 / (y.square().mean(1, keepdim=True) + EPS).sqrt() if post else 1.0
    add = scale * gate_of(d, seq, T) * y * k * gp
    r = x + add
    rb = B if d["x"].dtype == BF else U
    ek = rel_k(H) if post else 0.0
    near(f["r"][m], r[m], (rb * r.abs() + (1 + B) * (ek + 16 * U) * add.abs() + 2 * U * r.abs())[m], "r")
    if post:
        near(f["rstd_post"][m], k[m, 0], ek * k[m, 0], "rstd_post")
    if nxt:
        rr = f["r"].to(F64)                          # the norm of what is stored
        k = 1 / (rr.square().mean(1, keepdim=True) + EPS).sqrt()
        xn = rr * k * d["gn"].to(F64)
        near(f["xn"][m], xn[m], ((B + 2 * rel_k(H) + 16 * U) * xn.abs())[m], "xn")
        near(f["rstd_next"][m], k[m, 0], rel_k(H) * k[m, 0], "rstd_next")


def check_backward(d, seq, saved, g, scale, post, nxt, with_dr=True):
    T, H = d["x"].shape
    m = rows_in(seq, T)
    r, y, d_xn = saved["r"].to(F64), d["y"].to(F64), d["d_xn"].to(F64)
    gate, gp, gn = gate_of(d, seq, T), d["gp"].to(F64) if post else 1.0, d["gn"].to(F64)
    ts = 2 * (H / 256 + 24) * U                      # a row's sum
    cols = 2 * (T / 300 + 320) * U                   # a column's
    dx = d["d_r"].to(F64) if with_dr else torch.zeros_like(r)
    ex = 2 * U * dx.abs()
    if nxt:
        k = saved["rstd_next"].to(F64)[:, None]
        rh, t = r * k, d_xn * gn
        mean = (t * rh).mean(1, keepdim=True)
        ab = (t * rh).abs().mean(1, keepdim=True)
        dx = dx + k * (t - rh * mean)
        ex = ex + 16 * U * (dx.abs() + k * (t.abs() + rh.abs() * mean.abs())) + \
            k * rh.abs() * ab * (ts + 16 * U)
        v = (d_xn * rh)[m]
        near(g["d_gamma_next"], v.sum(0), (cols + 4 * U) * v.abs().sum(0), "d_gamma_next")
    rb = B if d["x"].dtype == BF else U
    near(g["d_x"][m], dx[m], (ex + rb * dx.abs())[m], "d_x")
    k = saved["rstd_post"].to(F64)[:, None] if post else 1.0
    yh = y * k
    q = scale * dx * gate * gp
    eq = abs(scale) * ex * (gate * torch.ones_like(y)).abs() * (gp if post else 1.0) + 8 * U * q.abs()
    if post:
        mean, ab = (q * yh).mean(1, keepdim=True), (q * yh).abs().mean(1, keepdim=True)
        dy = k * (q - yh * mean)
        ey = k * (eq + yh.abs() * ((eq * yh.abs()).mean(1, keepdim=True) + ab * (ts + 16 * U)) +
                  16 * U * (q.abs() + yh.abs() * mean.abs()))
    else:
        dy, ey = q, eq
    yb = B if d["y"].dtype == BF else U
    near(g["d_y"][m], dy[m], (ey * (1 + B) + yb * dy.abs())[m], "d_y")
    S = len(seq) - 1 if seq and d["gate"] is not None else 1
    b = seq if seq and d["gate"] is not None else [0, T]
    tot, et = torch.zeros(H, dtype=F64, device=DEV), torch.zeros(H, dtype=F64, device=DEV)
    for s in range(S):
        w = slice(b[s], b[s + 1])
        c = (scale * dx[w] * yh[w]).sum(0)
        e = (abs(scale) * ex[w] * yh[w].abs()).sum(0) + (cols + 8 * U) * (scale * dx[w] * yh[w]).abs().sum(0)
        if d["gate"] is not None:
            near(g["d_gate"][s], gp * c, (gp * torch.ones_like(e)).abs() * e + 2 * U * c.abs() * abs(1.0),
                 "d_gate")
            gs = d["gate"][s].to(F64)
            tot, et = tot + gs * c, et + gs.abs() * e + (S + 2) * U * (gs * c).abs()
        else:
            tot, et = tot + c, et + e
    if post:
        near(g["d_gamma_post"], tot, et, "d_gamma_post")


CASES = [(1, 8, None), (1, 4096, None), (3, 64, [0, 1, 3]), (37, 264, [0, 0, 20, 20, 37]),
         (300, 512, [5, 100, 290]), (700, 1024, [0, 350, 700]), (1000, 2048, None), (611, 2056, [0, 611]),
         (333, 4096, [0, 1, 2, 200, 333]), (50, 8192, [3, 3, 40, 44]), (2500, 256, list(range(0, 2501, 100))),
         (5000, 96, [0] + [17 * i for i in range(1, 200)]), (40, 8184, None)]


@pytest.mark.parametrize("T,H,seq", CASES)
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_forward_and_backward(T, H, seq, xt, yt):
    d = make(T, H, seq, T + H, xt, yt)
    st = moe.new_status(DEV)
    kw = dict(gamma_post=d["gp"], gate=d["gate"], scale=0.7, gamma_next=d["gn"], seq_offsets=d["seq"],
              status=st)
    f = moe.norm_residual(d["x"], d["y"], eps=EPS, **kw)
    check_forward(d, seq, f, 0.7, True, True)
    g = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, **kw)
    check_backward(d, seq, f, g, 0.7, True, True)
    assert int(st.item()) == 0


@pytest.mark.parametrize("post,nxt,gated,with_dr", [(False, True, True, True), (True, False, True, True),
                                                    (True, True, False, True), (True, True, True, False),
                                                    (False, False, False, True), (False, True, False, False)])
def test_parts(post, nxt, gated, with_dr):
    T, H, seq = 200, 1536, [0, 90, 200]
    d = make(T, H, seq, 1, F32, BF, gated)
    kw = dict(gamma_post=d["gp"] if post else None, gate=d["gate"], scale=-1.3,
              gamma_next=d["gn"] if nxt else None, post_norm=post, seq_offsets=d["seq"])
    f = moe.norm_residual(d["x"], d["y"], next_norm=nxt, eps=EPS, **kw)
    assert (f["xn"] is None) == (not nxt) and (f["rstd_post"] is None) == (not post)
    check_forward(d, seq if gated else None, f, -1.3, post, nxt)
    g = moe.norm_residual_backward(d["d_r"] if with_dr else None, d["d_xn"] if nxt else None, d["y"], f, **kw)
    assert (g["d_gate"] is None) == (not gated) and (g["d_gamma_next"] is None) == (not nxt)
    check_backward(d, seq if gated else None, f, g, -1.3, post, nxt, with_dr)


def test_plain_gammas_are_ones():
    d = make(20, 256, None, 2)
    one = torch.ones(256, dtype=BF, device=DEV)
    a = moe.norm_residual(d["x"], d["y"])
    b = moe.norm_residual(d["x"], d["y"], gamma_post=one, gamma_next=one, gate=one[None].contiguous())
    for k in a:
        assert torch.equal(a[k], b[k])


def test_rows_outside_every_sequence_are_left():
    T, H, seq = 30, 512, [4, 9, 9, 21]
    d = make(T, H, seq, 3)
    want = moe.norm_residual(d["x"], d["y"], gamma_post=d["gp"], gate=d["gate"], gamma_next=d["gn"],
                             seq_offsets=d["seq"])
    for t in ("x", "y", "d_r", "d_xn"):
        d[t][:4] = float("nan")
        d[t][21:] = float("nan")
    f = moe.norm_residual(d["x"], d["y"], gamma_post=d["gp"], gate=d["gate"], gamma_next=d["gn"],
                          seq_offsets=d["seq"])
    for k in f:
        assert torch.equal(f[k][4:21], want[k][4:21])
    # in place over marked buffers, through the C entry points
    import ctypes
    L, p = moe.lib(), lambda t: ctypes.c_void_p(t.data_ptr())            # noqa: E731
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    r, xn = (torch.full((T, H), 7.0, dtype=BF, device=DEV) for _ in range(2))
    kp, kn = (torch.full((T,), 7.0, device=DEV) for _ in range(2))
    assert L.moe_norm_residual(p(d["x"]), p(d["y"]), p(d["gp"]), p(d["gate"]), p(d["seq"]), 3, p(d["gn"]), T, H,
                               1.0, 1e-6, moe.POST_NORM, p(r), p(xn), p(kp), p(kn), None, s) == 0
    for t in (r, xn, kp, kn):
        assert (t[:4] == 7.0).all() and (t[21:] == 7.0).all() and torch.isfinite(t).all()
    g = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], dict(r=r, rstd_post=kp, rstd_next=kn),
                                   gamma_post=d["gp"], gate=d["gate"], gamma_next=d["gn"], seq_offsets=d["seq"])
    for k in ("d_gamma_post", "d_gamma_next", "d_gate"):
        assert torch.isfinite(g[k]).all()
    assert not g["d_gate"][1].any()                  # a sequence without tokens


def test_in_place():
    d = make(77, 1024, [0, 30, 77], 4)
    kw = dict(gamma_post=d["gp"], gate=d["gate"], gamma_next=d["gn"], seq_offsets=d["seq"])
    f = moe.norm_residual(d["x"], d["y"], **kw)
    want = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, **kw)
    import ctypes
    L, p = moe.lib(), lambda t: ctypes.c_void_p(t.data_ptr())            # noqa: E731
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    x, y, d_r = d["x"].clone(), d["y"].clone(), d["d_r"].clone()
    xn, kp, kn = torch.empty_like(x), torch.empty(77, device=DEV), torch.empty(77, device=DEV)
    assert L.moe_norm_residual(p(x), p(y), p(d["gp"]), p(d["gate"]), p(d["seq"]), 2, p(d["gn"]), 77, 1024, 1.0, 1e-6,
                               moe.POST_NORM, p(x), p(xn), p(kp), p(kn), None, s) == 0
    assert torch.equal(x, f["r"]) and torch.equal(xn, f["xn"])
    assert L.moe_norm_residual_backward(p(d_r), p(d["d_xn"]), p(y), p(x), p(kp), p(kn), p(d["gp"]), p(d["gate"]),
                                        p(d["seq"]), 2, p(d["gn"]), 77, 1024, 1.0, moe.POST_NORM, p(d_r), p(y),
                                        None, None, None, None, 0, None, s) == 0
    assert torch.equal(d_r, want["d_x"]) and torch.equal(y, want["d_y"])


@pytest.mark.parametrize("seq", [[0, 5, 3], [-1, 4, 8], [0, 4, 9]])
def test_bad_bounds_write_nothing(seq):
    d = make(8, 256, [0, 4, 8], 5)
    bad = torch.tensor(seq, dtype=torch.int32, device=DEV)
    st = moe.new_status(DEV)
    moe.norm_residual(d["x"], d["y"], gate=d["gate"], seq_offsets=bad, status=st)
    assert int(st.item()) == moe.DEV_BAD_OFFSETS
    f = moe.norm_residual(d["x"], d["y"], gate=d["gate"], seq_offsets=d["seq"])
    st.zero_()
    moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, gate=d["gate"], seq_offsets=bad, status=st)
    assert int(st.item()) == moe.DEV_BAD_OFFSETS


def test_no_rows_and_zero_rows():
    d = make(0, 256, None, 6)
    f = moe.norm_residual(d["x"], d["y"], gate=d["gate"])
    g = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, gate=d["gate"])
    assert f["r"].shape == (0, 256) and not g["d_gate"].any() and not g["d_gamma_post"].any()
    d = make(9, 256, None, 7)
    d["x"].zero_()
    d["y"].zero_()
    f = moe.norm_residual(d["x"], d["y"])
    assert not f["r"].any() and not f["xn"].any()
    # 1 / sqrt(eps): eps as fp32, the root and the quotient round by u each, half of
    # the first's error reaching the result
    assert ((f["rstd_post"].to(F64) - 1000.0).abs() <= 3 * U * 1000.0).all()
    g = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f)
    assert all(torch.isfinite(v).all() for v in g.values() if v is not None)


def test_against_differences():
    """Directional differences of sum(d_r r + d_xn xn) in float64; fp32
    streams.  d_xn's gammas and y are bf16, exact in float64; what is left is the
    fp32 arithmetic, far below the differences' own error (1e-6 of the norms)."""
    T, H, seq = 40, 512, [0, 15, 40]
    d = make(T, H, seq, 8, F32, F32)
    kw = dict(gamma_post=d["gp"], gate=d["gate"], scale=0.6, gamma_next=d["gn"], seq_offsets=d["seq"])
    f = moe.norm_residual(d["x"], d["y"], eps=EPS, **kw)
    g = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, **kw)

    def loss(x, y, gp, gn, gate):
        k = 1 / (y.square().mean(1, keepdim=True) + EPS).sqrt()
        gt = torch.cat((gate[0].expand(15, H), gate[1].expand(25, H)))
        r = x + 0.6 * gt * y * k * gp
        xn = r / (r.square().mean(1, keepdim=True) + EPS).sqrt() * gn
        return float((d["d_r"].to(F64) * r).sum() + (d["d_xn"].to(F64) * xn).sum())

    p = [d[k].to(F64) for k in ("x", "y", "gp", "gn", "gate")]
    for i, k in enumerate(("d_x", "d_y", "d_gamma_post", "d_gamma_next", "d_gate")):
        v = torch.randn(p[i].shape, generator=torch.Generator().manual_seed(i)).to(F64).to(DEV)
        up, dn = list(p), list(p)
        up[i], dn[i] = p[i] + 1e-5 * v, p[i] - 1e-5 * v
        diff = (loss(*up) - loss(*dn)) / 2e-5
        got = g[k].to(F64)
        assert abs(float((got * v).sum()) - diff) <= 1e-5 * float(got.norm() * v.norm()), k


def test_captured_replayed_and_on_another_stream():
    d = make(500, 1024, [0, 100, 500], 9)
    kw = dict(gamma_post=d["gp"], gate=d["gate"], gamma_next=d["gn"], seq_offsets=d["seq"])

    def step():
        f = moe.norm_residual(d["x"], d["y"], **kw)
        g = moe.norm_residual_backward(d["d_r"], d["d_xn"], d["y"], f, **kw)
        return [*f.values(), *g.values()]

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    d["y"].copy_(d["y"].roll(3, 0))
    d["seq"].copy_(torch.tensor([0, 333, 500], dtype=torch.int32))
    want = step()
    for _ in range(2):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, cap))


def test_around_the_layer():
    """xn goes into the layer (without its own norm) as its RMSNorm would give
    it: the two agree to a last bf16 place, where the exact sum of squares and the
    fp32 one round apart."""
    T, H = 64, 256
    d = make(T, H, None, 10)
    f = moe.norm_residual(d["x"], d["y"], gamma_post=d["gp"], gamma_next=d["gn"])
    xn, _ = moe.rmsnorm_gate(f["r"], None, gamma=d["gn"])
    err = (xn.to(F64) - f["xn"].to(F64)).abs()
    assert (err <= 2 * B * xn.to(F64).abs()).all()
    assert (err > 0).float().mean() < 0.01
