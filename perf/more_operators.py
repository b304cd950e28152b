"""What the gated block's operators are measured on: its training passes, the
norms around it, and its products with 4-bit weights under bf16 rows.

Each case is one pass through an operator at one size; ``run`` makes it either
with the library's entry points (``own``) or in the plain form below, which is
written from the definitions with elementary torch operations.

Operators ("op" of a case), group g owning rows [offsets[g], offsets[g+1]):
  mlp_fwd    grouped_mlp_train: h = [gate up] = x W13[g]^T (kept for the
             backward pass), y = (SiLU(gate) up) W2[g]^T.
  mlp_bwd    grouped_mlp_backward: with d_act = d_y W2[g], s = sigmoid(gate),
               d_up = d_act gate s,  d_gate = d_act up s (1 + gate (1 - s)),
               d_x = [d_gate d_up] W13[g],
               d_W13[g] = [d_gate d_up]^T x,  d_W2[g] = d_y^T (SiLU(gate) up).
  norm_fwd   norm_residual: with N(v; gamma) = gamma v / sqrt(mean(v^2) + eps),
               r = x + scale gate[s] N(y; gamma_post),  xn = N(r; gamma_next)
             for the tokens of sequence s.
  norm_bwd   norm_residual_backward: the gradients of x, y, both gammas and the
             gate from those of r and xn, at the r that was kept.
  w4         fp4_weight_matmul and fp4_weight_swiglu: bf16 rows times 4-bit
             weights, y = x W[g]^T or SiLU(x Wg^T) (x Wu^T).

4-bit weights: e2m1 elements, two to a byte (the lower column in the low four
bits), one scale byte per 32 columns ("mx", 2^(b - 127)) or 16 ("nv", e4m3, and
a factor 2^scale_exp of the whole matrix).  The scale bytes lie in 512-byte
tiles of 128 rows x 4 blocks: row r, block b at (r % 32) * 16 + (r // 32) * 4 + b.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = {"mx": 32, "nv": 16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest block's training step: 128 rows on 8 experts, where the
        # launches count
        dict(name="mlp-forward-tiny", op="mlp_fwd", n=128, H=128, I=256, G=8, active=8, skew=0.0),
        # an image-generation block's batch, 16384 tokens on 8 of 64 experts each
        dict(name="mlp-forward-image", op="mlp_fwd", n=131072, H=4096, I=2048, G=64, active=64,
             skew=0.1),
        # fine-tuning on a handful of tokens: every gradient of every expert
        # has to be written, idle experts' included
        dict(name="mlp-backward-few", op="mlp_bwd", n=509, H=2048, I=1024, G=64, active=53,
             skew=0.5),
        # a batch of 4096 tokens on narrow experts, unevenly loaded
        dict(name="mlp-backward-batch", op="mlp_bwd", n=32768, H=2048, I=1024, G=64, active=61,
             skew=0.5),
        # the image-generation block's gradients
        dict(name="mlp-backward-image", op="mlp_bwd", n=131072, H=4096, I=2048, G=64, active=64,
             skew=0.1),
        # one token on its way through a decoder
        dict(name="norm-token", op="norm_fwd", T=1, H=4096, S=1, gated=True, f32=False),
        # the image-generation block's batch, four images with a gate each
        dict(name="norm-image", op="norm_fwd", T=16384, H=4096, S=4, gated=True, f32=False),
        dict(name="norm-backward-image", op="norm_bwd", T=16384, H=4096, S=4, gated=True,
             f32=False),
        # a packed batch of ragged sequences, one of them empty, the residual
        # stream in fp32
        dict(name="norm-backward-packed", op="norm_bwd", T=50021, H=2048, S=9, gated=True,
             f32=True),
        # decoding one token: a row for each of 8 experts
        dict(name="w4-token", op="w4", n=8, K=4096, N=2048, G=64, active=8, fmt="mx",
             swiglu=True, f32=False),
        # the shared expert for four tokens: one group of few rows
        dict(name="w4-shared", op="w4", n=4, K=4096, N=2048, G=1, active=1, fmt="nv",
             swiglu=True, f32=False),
        # the down projection of a decoding batch of 32 tokens
        dict(name="w4-decode", op="w4", n=256, K=2048, N=4096, G=64, active=63, fmt="nv",
             swiglu=False, f32=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mlp_fwd", "mlp_bwd", "mlp_bwd", "norm_fwd", "norm_bwd", "w4", "w4"])
    if op in ("norm_fwd", "norm_bwd"):
        H = 8 * _log(rng, 8, 1024)
        f32 = rng.random() < 0.4
        return dict(op=op, T=_log(rng, 1, 16384 * 4096 // (H * (2 if f32 else 1))), H=H,
                    S=rng.randint(1, 12), gated=rng.random() < 0.7, f32=f32)
    G = _log(rng, 1, 128)
    if op == "w4":
        K, N = 128 * _log(rng, 1, 40), 128 * _log(rng, 1, 32)
        while G * K * N > 64 * 4096 * 4096 // 2:
            G = max(1, G // 2)
        n = _log(rng, 1, 512)
        return dict(op=op, n=n, K=K, N=N, G=G, active=rng.randint(1, min(n, G)),
                    fmt=rng.choice(["mx", "nv"]), swiglu=rng.random() < 0.5,
                    f32=rng.random() < 0.3)
    H, I = 128 * _log(rng, 1, 40), 128 * _log(rng, 1, 24)
    while G * H * I > 64 * 4096 * 2048:
        G = max(1, G // 2)
    n = _log(rng, 1, min(131072, 131072 * 4096 * 2048 // (H * I)))
    return dict(op=op, n=n, H=H, I=I, G=G, active=rng.randint(1, min(n, G)),
                skew=rng.choice([0.0, 0.3, 1.0]))


# ------------------------------------------------------------------ inputs
def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + stream)
    return g


def _cpu_gen(seed, stream):
    g = torch.Generator()
    g.manual_seed(seed * 1000003 + stream)
    return g


def _normal(shape, sigma, gen, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEV) * sigma).to(dtype)


def _weights(G, rows, cols, gen):
    w = torch.empty((G, rows, cols), dtype=torch.bfloat16, device=DEV)
    for g in range(G):
        w[g] = _normal((rows, cols), 0.02, gen)
    return w


def _offsets(case, seed):
    """Rows of each group: exactly `active` groups have any, sizes fall off
    as rank^-skew."""
    n, G, a = case["n"], case["G"], case["active"]
    g = _cpu_gen(seed, 4)
    who = torch.randperm(G, generator=g)[:a]
    p = torch.arange(1, a + 1, dtype=torch.float64) ** -case.get("skew", 0.0)
    extra = torch.bincount(torch.multinomial(p, max(n - a, 1), replacement=True, generator=g)
                           if n > a else torch.zeros(0, dtype=torch.int64), minlength=a)
    counts = torch.zeros(G, dtype=torch.int64)
    counts[who] = 1 + extra
    off = torch.zeros(G + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(counts, 0)
    return off.to(DEV)


def _sequences(T, S, seed):
    """S + 1 ascending token bounds; of three or more sequences the second is
    empty."""
    cuts = torch.randint(0, T + 1, (S - 1,), generator=_cpu_gen(seed, 3)).sort().values.tolist()
    b = [0] + cuts + [T]
    if S >= 3:
        b[2] = b[1]
    return b


def _quantized_weights(G, rows, K, fmt, scale_exp, gen):
    """Packed codes [G, rows, K/2] and scale tiles of normal weights."""
    q = torch.empty((G, rows, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((G * rows, K // BLOCK[fmt]), dtype=torch.uint8, device=DEV)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for g in range(G):
        f = _normal((rows, K), 0.02, gen).to(torch.float32).view(rows, -1, BLOCK[fmt])
        amax = f.abs().amax(2)
        if fmt == "mx":
            b = (torch.frexp(amax)[1] - 3 + 127).clamp(0, 254)
            v = f * torch.exp2(127.0 - b)[:, :, None]
        else:
            s8 = (amax / 6.0 * 2.0 ** -scale_exp).clamp(max=448.0).to(torch.float8_e4m3fn)
            b = s8.view(torch.uint8)
            v = f / (s8.to(torch.float32) * 2.0 ** scale_exp).clamp(min=1e-30)[:, :, None]
        c = torch.bucketize(v.abs(), mids).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
        c = c.view(rows, K)
        q[g] = c[:, 0::2] | (c[:, 1::2] << 4)
        s[g * rows:(g + 1) * rows] = b.to(torch.uint8)
    # [row block, 4, 32, block of 4, 4] -> [row block, block of 4, 32, 4, 4]
    tiles = s.view(G * rows // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4)
    return q, tiles.reshape(-1).contiguous()


def prepare(case, seed):
    op = case["op"]
    st = dict(case=case)
    if op in ("mlp_fwd", "mlp_bwd"):
        n, H, I, G = case["n"], case["H"], case["I"], case["G"]
        st.update(offsets=_offsets(case, seed), x=_normal((n, H), 1.0, _gen(seed, 10)),
                  w13=_weights(G, 2 * I, H, _gen(seed, 11)),
                  w2=_weights(G, H, I, _gen(seed, 12)))
        if op == "mlp_bwd":
            # what the forward pass kept: x W13^T has about this spread
            st.update(h=_normal((n, 2 * I), 0.02 * math.sqrt(H), _gen(seed, 13)),
                      d_y=_normal((n, H), 1e-2, _gen(seed, 14)))
    elif op in ("norm_fwd", "norm_bwd"):
        T, H, S = case["T"], case["H"], case["S"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        st.update(y=_normal((T, H), 0.7, _gen(seed, 20)),
                  gamma_post=_normal((H,), 0.1, _gen(seed, 21)) + 1.0,
                  gamma_next=_normal((H,), 0.1, _gen(seed, 22)) + 1.0, scale=0.5,
                  gate=_normal((S, H), 0.5, _gen(seed, 23)) if case["gated"] else None,
                  seq=torch.tensor(_sequences(T, S, seed), dtype=torch.int32, device=DEV)
                  if S > 1 else None)
        stream = _normal((T, H), 2.0, _gen(seed, 24), dt)
        stream[:, ::61] *= 8.0               # a residual stream's outlier channels
        if op == "norm_fwd":
            st.update(x=stream)
        else:
            # what the forward pass kept, and the gradients that arrive
            ms = lambda v: v.to(torch.float64).square().mean(1)        # noqa: E731
            saved = dict(r=stream, rstd_post=(1.0 / (ms(st["y"]) + EPS).sqrt()).float(),
                         rstd_next=(1.0 / (ms(stream) + EPS).sqrt()).float())
            st.update(saved=saved, d_r=_normal((T, H), 1e-2, _gen(seed, 25), dt),
                      d_xn=_normal((T, H), 1e-2, _gen(seed, 26)))
    else:
        n, K, N, G, fmt = case["n"], case["K"], case["N"], case["G"], case["fmt"]
        we = 0 if fmt == "mx" else -6        # lifts weights of 0.02 into e4m3's range
        q, sf = _quantized_weights(G, 2 * N if case["swiglu"] else N, K, fmt, we, _gen(seed, 30))
        x = _normal((n, K), 1.0, _gen(seed, 31))
        x[:, ::97] *= 12.0                   # outlier channels
        st.update(offsets=_offsets(case, seed), x=x, w_q=q, w_sf=sf, w_exp=we)
    return st


# ------------------------------------------------------------------ plain form
def _groups(st):
    off = st["offsets"].tolist()
    return [(g, off[g], off[g + 1]) for g in range(len(off) - 1)]


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _plain_mlp_fwd(st):
    I = st["case"]["I"]
    h = torch.empty((st["x"].shape[0], 2 * I), dtype=torch.bfloat16, device=DEV)
    y = torch.empty_like(st["x"])
    for g, a, b in _groups(st):
        if a == b:
            continue
        v = st["x"][a:b].float() @ st["w13"][g].float().T
        h[a:b] = v.to(torch.bfloat16)
        act = _silu(v[:, :I]) * v[:, I:]
        y[a:b] = (act @ st["w2"][g].float().T).to(torch.bfloat16)
    return dict(h=h, y=y)


def _plain_mlp_bwd(st):
    I = st["case"]["I"]
    d_x = torch.empty_like(st["x"])
    d_w13 = torch.empty_like(st["w13"])
    d_w2 = torch.empty_like(st["w2"])
    for g, a, b in _groups(st):
        if a == b:
            d_w13[g].zero_()
            d_w2[g].zero_()
            continue
        x, d_y = st["x"][a:b].float(), st["d_y"][a:b].float()
        gate, up = st["h"][a:b, :I].float(), st["h"][a:b, I:].float()
        s = 1.0 / (1.0 + torch.exp(-gate))
        d_act = d_y @ st["w2"][g].float()
        d_h = torch.cat((d_act * up * s * (1.0 + gate * (1.0 - s)), d_act * gate * s), 1)
        d_x[a:b] = (d_h @ st["w13"][g].float()).to(torch.bfloat16)
        d_w13[g] = (d_h.T @ x).to(torch.bfloat16)
        d_w2[g] = (d_y.T @ (gate * s * up)).to(torch.bfloat16)
    return dict(d_x=d_x, d_w13=d_w13, d_w2=d_w2)


def _sequence_of(st, T):
    if st["seq"] is None:
        return torch.zeros(T, dtype=torch.int64, device=DEV)
    seq = st["seq"].long()
    return torch.searchsorted(seq[1:].contiguous(), torch.arange(T, device=DEV), right=True)


def _plain_norm_fwd(st):
    x, y = st["x"].float(), st["y"].float()
    n = y / (y.square().mean(1, keepdim=True) + EPS).sqrt() * st["gamma_post"].float()
    if st["gate"] is not None:
        n = n * st["gate"].float()[_sequence_of(st, x.shape[0])]
    r = (x + st["scale"] * n).to(st["x"].dtype)
    v = r.float()
    xn = v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * st["gamma_next"].float()
    return dict(r=r, xn=xn.to(torch.bfloat16))


def _plain_norm_bwd(st):
    sv = st["saved"]
    T, H = st["y"].shape
    S = st["case"]["S"]
    d_xn = st["d_xn"].float()
    rs = sv["rstd_next"][:, None]
    rhat = sv["r"].float() * rs
    t = d_xn * st["gamma_next"].float()
    d_r = st["d_r"].float() + rs * (t - rhat * (t * rhat).mean(1, keepdim=True))
    ys = sv["rstd_post"][:, None]
    yhat = st["y"].float() * ys
    sid = _sequence_of(st, T)
    gp = st["gamma_post"].float()
    sums = torch.zeros((S, H), dtype=torch.float64, device=DEV)
    sums.index_add_(0, sid, (st["scale"] * d_r * yhat).to(torch.float64))
    d_n = st["scale"] * d_r
    out = dict(d_x=d_r.to(sv["r"].dtype), d_gamma_next=(d_xn * rhat).to(torch.float64).sum(0).float())
    if st["gate"] is not None:
        gate = st["gate"].float()
        d_n = d_n * gate[sid]
        out["d_gate"] = (sums * gp).float()
        sums = sums * gate
    out["d_gamma_post"] = sums.sum(0).float()
    t = d_n * gp
    out["d_y"] = (ys * (t - yhat * (t * yhat).mean(1, keepdim=True))).to(torch.bfloat16)
    return out


def _plain_w4(st):
    c = st["case"]
    N, K, fmt = c["N"], c["K"], c["fmt"]
    rows = st["w_q"].shape[1]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    out = torch.empty((c["n"], N), dtype=torch.float32 if c["f32"] else torch.bfloat16, device=DEV)
    tiles = st["w_sf"].view(c["G"], rows // 128, -1, 32, 4, 4)
    for g, a, b in _groups(st):
        if a == b:
            continue
        q = st["w_q"][g]
        v = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), 2).view(rows, K)
        s = tiles[g].permute(0, 3, 2, 1, 4).reshape(rows, -1)
        if fmt == "mx":
            s = torch.exp2(s.float() - 127.0)
        else:
            s = s.view(torch.float8_e4m3fn).float() * 2.0 ** st["w_exp"]
        w = (v.view(rows, -1, BLOCK[fmt]) * s[:, :, None]).view(rows, K)
        y = st["x"][a:b].float() @ w.T
        if c["swiglu"]:
            y = _silu(y[:, :N]) * y[:, N:]
        out[a:b] = y.to(out.dtype)
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return {"mlp_fwd": _plain_mlp_fwd, "mlp_bwd": _plain_mlp_bwd, "norm_fwd": _plain_norm_fwd,
                "norm_bwd": _plain_norm_bwd, "w4": _plain_w4}[op](state)
    import moe_expert_routing_fp32_gb300 as moe
    if op == "mlp_fwd":
        h, y = moe.grouped_mlp_train(state["x"], state["offsets"], state["w13"], state["w2"])
        return dict(h=h, y=y)
    if op == "mlp_bwd":
        d_x, d_w13, d_w2 = moe.grouped_mlp_backward(state["d_y"], state["x"], state["offsets"],
                                                    state["h"], state["w13"], state["w2"])
        return dict(d_x=d_x, d_w13=d_w13, d_w2=d_w2)
    if op == "norm_fwd":
        f = moe.norm_residual(state["x"], state["y"], gamma_post=state["gamma_post"],
                              gamma_next=state["gamma_next"], gate=state["gate"],
                              scale=state["scale"], eps=EPS, seq_offsets=state["seq"])
        return dict(r=f["r"], xn=f["xn"])
    if op == "norm_bwd":
        d = moe.norm_residual_backward(state["d_r"], state["d_xn"], state["y"], state["saved"],
                                       gamma_post=state["gamma_post"],
                                       gamma_next=state["gamma_next"], gate=state["gate"],
                                       scale=state["scale"], seq_offsets=state["seq"])
        out = dict(d_x=d["d_x"], d_gamma_next=d["d_gamma_next"])
        if c["gated"]:
            out["d_gate"] = d["d_gate"]
        out.update(d_gamma_post=d["d_gamma_post"], d_y=d["d_y"])
        return out
    w = moe.Fp4Matrix(state["w_q"], state["w_sf"], c["fmt"], state["w_exp"])
    f = moe.fp4_weight_swiglu if c["swiglu"] else moe.fp4_weight_matmul
    return f(state["x"], state["offsets"], w, out_f32=c["f32"])


# ------------------------------------------------------------------ floors
def work(case):
    op = case["op"]
    if op in ("mlp_fwd", "mlp_bwd"):
        n, H, I, G, a = case["n"], case["H"], case["I"], case["G"], case["active"]
        w = 3 * H * I * 2
        if op == "mlp_fwd":
            return {"bytes": n * (4 * H + 4 * I) + a * w, "flops": 6 * n * H * I}
        return {"bytes": n * (6 * H + 4 * I) + (a + G) * w, "flops": 12 * n * H * I}
    if op in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        e = 4 if case["f32"] else 2
        if op == "norm_fwd":
            return {"bytes": T * H * (2 * e + 4), "flops": 12 * T * H}
        return {"bytes": T * H * (3 * e + 6), "flops": 30 * T * H}
    n, K, N = case["n"], case["K"], case["N"]
    rows = 2 * N if case["swiglu"] else N
    per = 0.5 + 1.0 / BLOCK[case["fmt"]]
    return {"bytes": int(case["active"] * rows * K * per) + n * K * 2 +
            n * N * (4 if case["f32"] else 2), "flops": 2 * n * K * rows}


# ------------------------------------------------------------------ 64 bits
def _exact_values(q, s, fmt, scale_exp):
    out = torch.empty((q.shape[0], q.shape[1] * 2), dtype=torch.float64, device=DEV)
    for half, c in ((0, q & 15), (1, q >> 4)):
        c = c.to(torch.int32)
        e, m = (c >> 1) & 3, (c & 1).to(torch.float64)
        mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((e - 1).to(torch.float64)))
        out[:, half::2] = torch.where(c >= 8, -mag, mag)
    b = s.to(torch.int32)
    if fmt == "mx":
        sv = torch.exp2((b - 127).to(torch.float64))
    else:
        e, m = (b >> 3) & 15, (b & 7).to(torch.float64)
        sv = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8) * torch.exp2((e - 7).to(torch.float64)))
        sv = sv * 2.0 ** scale_exp
    return out * sv.repeat_interleave(BLOCK[fmt], dim=1)


def _spans(st, T):
    """(sequence, first token, end) of every sequence that has tokens."""
    b = [0, T] if st["seq"] is None else st["seq"].tolist()
    return [(s, b[s], b[s + 1]) for s in range(len(b) - 1) if b[s + 1] > b[s]]


def exact(case, seed):
    op = case["op"]
    if op.startswith("mlp") and work(case)["flops"] > 7e12:
        return None                          # a minute of 64-bit products
    st = prepare(case, seed)
    f64 = torch.float64
    if op == "mlp_fwd":
        n, H, I = case["n"], case["H"], case["I"]
        h = torch.empty((n, 2 * I), dtype=f64, device=DEV)
        y = torch.empty((n, H), dtype=f64, device=DEV)
        for g in range(case["G"]):
            a, b = int(st["offsets"][g]), int(st["offsets"][g + 1])
            if b > a:
                torch.mm(st["x"][a:b].to(f64), st["w13"][g].to(f64).T, out=h[a:b])
                act = h[a:b, :I] * torch.sigmoid(h[a:b, :I]) * h[a:b, I:]
                torch.mm(act, st["w2"][g].to(f64).T, out=y[a:b])
        return dict(h=h, y=y)
    if op == "mlp_bwd":
        n, H, I, G = case["n"], case["H"], case["I"], case["G"]
        d_x = torch.empty((n, H), dtype=f64, device=DEV)
        d_w13 = torch.zeros((G, 2 * I, H), dtype=f64, device=DEV)
        d_w2 = torch.zeros((G, H, I), dtype=f64, device=DEV)
        for g in range(G):
            a, b = int(st["offsets"][g]), int(st["offsets"][g + 1])
            if b == a:
                continue
            h = st["h"][a:b].to(f64).requires_grad_()
            with torch.enable_grad():
                gate, up = h.chunk(2, 1)
                act = gate * torch.sigmoid(gate) * up
            dy = st["d_y"][a:b].to(f64)
            d_h, = torch.autograd.grad(act, h, dy @ st["w2"][g].to(f64))
            torch.mm(dy.T, act.detach(), out=d_w2[g])
            torch.mm(d_h, st["w13"][g].to(f64), out=d_x[a:b])
            torch.mm(d_h.T, st["x"][a:b].to(f64), out=d_w13[g])
        return dict(d_x=d_x, d_w13=d_w13, d_w2=d_w2)
    if op in ("norm_fwd", "norm_bwd"):
        T, H = case["T"], case["H"]
        gp, gn = st["gamma_post"].to(f64), st["gamma_next"].to(f64)
        one = torch.ones(H, dtype=f64, device=DEV)
        out = {}
        if op == "norm_fwd":
            out = dict(r=torch.empty((T, H), dtype=f64, device=DEV),
                       xn=torch.empty((T, H), dtype=f64, device=DEV))
        else:
            out = dict(d_x=torch.empty((T, H), dtype=f64, device=DEV),
                       d_gamma_next=torch.zeros(H, dtype=f64, device=DEV))
            if case["gated"]:
                out["d_gate"] = torch.zeros((case["S"], H), dtype=f64, device=DEV)
            out.update(d_gamma_post=torch.zeros(H, dtype=f64, device=DEV),
                       d_y=torch.empty((T, H), dtype=f64, device=DEV))
        for s, a, b in _spans(st, T):
            gate = st["gate"][s].to(f64) if case["gated"] else one
            for i in range(a, b, 8192):
                j = min(b, i + 8192)
                y = st["y"][i:j].to(f64)
                if op == "norm_fwd":
                    rms = torch.sqrt(torch.einsum("th,th->t", y, y) / H + EPS)
                    r = st["x"][i:j].to(f64) + st["scale"] * gate * gp * (y / rms[:, None])
                    out["r"][i:j] = r
                    rms = torch.sqrt(torch.einsum("th,th->t", r, r) / H + EPS)
                    out["xn"][i:j] = r / rms[:, None] * gn
                    continue
                # the norms' Jacobians at the values that were kept: for
                # N(v) = k v with k = 1 / rms(v),  d_v = k d_N - k^3 v <v, d_N> / H
                r, dn = st["saved"]["r"][i:j].to(f64), st["d_xn"][i:j].to(f64)
                k = torch.rsqrt(torch.einsum("th,th->t", r, r) / H + EPS)[:, None]
                dot = torch.einsum("th,th->t", r, dn * gn)[:, None]
                d_r = st["d_r"][i:j].to(f64) + k * dn * gn - k ** 3 * r * dot / H
                out["d_x"][i:j] = d_r
                out["d_gamma_next"] += (dn * r * k).sum(0)
                k = torch.rsqrt(torch.einsum("th,th->t", y, y) / H + EPS)[:, None]
                c = st["scale"] * torch.einsum("th,th->h", d_r, y * k)
                if case["gated"]:
                    out["d_gate"][s] += c * gp
                out["d_gamma_post"] += c * gate
                d_n = st["scale"] * gate * gp * d_r
                dot = torch.einsum("th,th->t", y, d_n)[:, None]
                out["d_y"][i:j] = k * d_n - k ** 3 * y * dot / H
        return out
    n, K, N, G, fmt = case["n"], case["K"], case["N"], case["G"], case["fmt"]
    rows = 2 * N if case["swiglu"] else N
    nb = K // BLOCK[fmt]
    r, b = torch.arange(rows, device=DEV), torch.arange(nb, device=DEV)
    at = ((r[:, None] // 128) * (nb // 4) + b // 4) * 512 + \
        ((r % 32) * 16 + (r % 128) // 32 * 4)[:, None] + b % 4
    out = torch.empty((n, N), dtype=f64, device=DEV)
    for g in range(G):
        a, e = int(st["offsets"][g]), int(st["offsets"][g + 1])
        if e <= a:
            continue
        s = st["w_sf"][g * rows * nb:(g + 1) * rows * nb][at]
        y = st["x"][a:e].to(f64) @ _exact_values(st["w_q"][g], s, fmt, st["w_exp"]).T
        out[a:e] = torch.sigmoid(y[:, :N]) * y[:, :N] * y[:, N:] if case["swiglu"] else y
    return out
