"""What the router's training operators and the 4-bit expert operators are
measured on.

Each case is one pass through an operator at one size; ``run`` makes it either
with the library's entry points (``own``) or in the plain form below, which is
written from the definitions with elementary torch operations.

Operators ("op" of a case):
  router     balance_loss and gate_topk_backward: the training step of the
             gate.  With p = softmax(logits[t]), c[s, e] the assignments of
             sequence s to expert e, n_s its unmasked tokens, S+ the sequences
             that have any:
               prob_mean[s, e] = (1 / n_s) sum_t p[t, e]
               loss = (coef / S+) sum_s E / (k n_s) sum_e c[s, e] prob_mean[s, e]
               d_logits[t, i] = coef E / (S+ k n_s^2) p_i (c[s, i] - sum_e p_e c[s, e])
                                + the gradient through the top-k weights;
             masked tokens take no part and get a zero gradient.
  combine    finalize_routing_backward: d_y_exp[row(t, j)] = w[t, j] d_out[t],
             d_topk_w[t, j] = <d_out[t], y_exp[row(t, j)]>.
  quantize   fp4_quantize of token rows into expert order, and fp4_dequantize:
             what the rows stand for afterwards.
  swiglu     fp4_grouped_swiglu: act = bf16(SiLU(g) u), [g u] = A W13[grp]^T on
             4-bit operands with fp32 accumulation.
  matmul     fp4_grouped_matmul: y = A W[grp]^T, bf16 or fp32.

4-bit operands: e2m1 elements, two to a byte (the lower index in the low four
bits), and one scale byte per block of 32 ("mx", a power of two, 2^(b - 127))
or 16 elements ("nv", e4m3); "nv" values carry a further factor
2^scale_exp of the whole matrix.  The scale bytes lie in 512-byte tiles of 128
rows x 4 blocks (see ``scale_index``); with groups, the tiles of group g start
at row block offsets[g] / 128 + g.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"mx": 32, "nv": 16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the gate of the smallest block while it is being trained: a few
        # microseconds of work, where the launches count
        dict(name="router-tiny", op="router", T=64, E=8, k=2, S=1, pad=0.0, renorm=True,
             weights=True),
        # an image-generation block's batch: four sequences, a tenth padding
        dict(name="router-image", op="router", T=16384, E=64, k=8, S=4, pad=0.1, renorm=True,
             weights=True),
        # a long packed batch on many experts, the loss alone; ragged sequences,
        # one of them empty and one with every token masked
        dict(name="router-packed", op="router", T=250007, E=160, k=6, S=9, pad=0.05, renorm=False,
             weights=False),
        # the weighted sum's gradients for a handful of tokens, fp32 rows
        dict(name="combine-few", op="combine", T=37, H=2048, E=16, k=8, f32=True),
        # and for the image-generation block
        dict(name="combine-image", op="combine", T=16384, H=4096, E=64, k=8, f32=False),
        # the token rows of a small serving batch to 4 bits, in expert order
        dict(name="quantize-small", op="quantize", T=64, K=4096, E=64, k=8, fmt="nv"),
        # and those of the image-generation block
        dict(name="quantize-image", op="quantize", T=16384, K=4096, E=64, k=8, fmt="mx"),
        # decoding eight tokens: 64 rows over 41 experts, all of it weights
        dict(name="swiglu-decode", op="swiglu", n=64, K=4096, N=2048, G=64, active=41, skew=0.0,
             fmt="mx", f32=False),
        # a batch of 4096 tokens on narrow experts, unevenly loaded
        dict(name="swiglu-batch", op="swiglu", n=32768, K=2048, N=1024, G=64, active=61, skew=0.5,
             fmt="nv", f32=False),
        # the image-generation block's experts, both products
        dict(name="swiglu-image", op="swiglu", n=131072, K=4096, N=2048, G=64, active=64, skew=0.1,
             fmt="mx", f32=False),
        dict(name="matmul-decode", op="matmul", n=512, K=2048, N=4096, G=64, active=63, skew=0.0,
             fmt="nv", f32=False),
        dict(name="matmul-image", op="matmul", n=131072, K=2048, N=4096, G=64, active=64, skew=0.1,
             fmt="nv", f32=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "combine", "quantize", "swiglu", "matmul", "swiglu", "matmul"])
    if op == "router":
        E = _log(rng, 4, 512)
        k = rng.randint(1, min(E, 12))
        T = _log(rng, 1, min(250000, 40_000_000 // E))
        return dict(op=op, T=T, E=E, k=k, S=rng.randint(1, 12), pad=rng.choice([0.0, 0.02, 0.3]),
                    renorm=rng.random() < 0.5, weights=rng.random() < 0.7)
    if op == "combine":
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(E, 10))
        H = 8 * _log(rng, 16, 1024)
        return dict(op=op, T=_log(rng, 1, 16384 * 8 * 4096 // (k * H * 2)), H=H, E=E, k=k,
                    f32=rng.random() < 0.4)
    if op == "quantize":
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(E, 10))
        K = 128 * _log(rng, 1, 48)
        return dict(op=op, T=_log(rng, 1, min(40000, 16384 * 8 * 4096 // (k * K))), K=K, E=E, k=k,
                    fmt=rng.choice(["mx", "nv"]))
    G = _log(rng, 1, 128)
    K = 128 * _log(rng, 1, 40)
    N = 128 * _log(rng, 1, 32)
    while G * K * N > 64 * 4096 * 4096 // 2:
        G = max(1, G // 2)
    n = _log(rng, 1, min(131072, 16384 * 4096 * 8 * 2048 // (K * N)))
    return dict(op=op, n=n, K=K, N=N, G=G, active=rng.randint(1, min(n, G)),
                skew=rng.choice([0.0, 0.3, 1.0]), fmt=rng.choice(["mx", "nv"]),
                f32=op == "matmul" and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + stream)
    return g


def _cpu_gen(seed, stream):
    g = torch.Generator()
    g.manual_seed(seed * 1000003 + stream)
    return g


def _logits(T, E, seed):
    """Gate logits with a tilt between experts, as a router has early on."""
    lg = torch.randn((T, E), generator=_gen(seed, 1), device=DEV)
    return lg * 1.3 + 0.4 * torch.randn((1, E), generator=_gen(seed, 2), device=DEV)


def _routing(T, E, k, seed):
    """Assignments of T tokens and their rows in expert order (stable)."""
    lg = _logits(T, E, seed)
    w, idx = torch.topk(torch.softmax(lg, 1), k, dim=1)
    w = w / w.sum(1, keepdim=True)
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    row_idx = torch.empty_like(order)
    row_idx[order] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    return lg, idx.to(torch.int32), w, row_idx.to(torch.int32), offsets


def _sequences(T, S, seed):
    """S + 1 ascending token bounds; with three or more sequences the second
    one is empty and (see prepare) the third one entirely masked."""
    cuts = torch.randint(0, T + 1, (S - 1,), generator=_cpu_gen(seed, 3)).sort().values.tolist()
    b = [0] + cuts + [T]
    if S >= 3:
        b[2] = b[1]
    return b


def _offsets(case, seed):
    """Rows of each group: exactly `active` groups have any, sizes fall off
    as rank^-skew."""
    n, G, a = case["n"], case["G"], case["active"]
    g = _cpu_gen(seed, 4)
    who = torch.randperm(G, generator=g)[:a]
    p = torch.arange(1, a + 1, dtype=torch.float64) ** -case["skew"]
    extra = torch.bincount(torch.multinomial(p, max(n - a, 1), replacement=True, generator=g)
                           if n > a else torch.zeros(0, dtype=torch.int64), minlength=a)
    counts = torch.zeros(G, dtype=torch.int64)
    counts[who] = 1 + extra
    off = torch.zeros(G + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(counts, 0)
    return off.to(DEV)


def _normal(shape, sigma, gen):
    return (torch.randn(shape, generator=gen, device=DEV) * sigma).to(torch.bfloat16)


def prepare(case, seed):
    op = case["op"]
    st = dict(case=case)
    if op == "router":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        lg, idx, _, _, _ = _routing(T, E, k, seed)
        bounds = _sequences(T, S, seed)
        mask = torch.rand(T, generator=_gen(seed, 5), device=DEV) >= case["pad"]
        if S >= 3:
            mask[bounds[2]:bounds[3]] = False
        lg[~mask] = float("nan")            # whatever padding holds
        st.update(logits=lg, idx=idx, coef=0.01,
                  mask=mask.to(torch.uint8) if case["pad"] > 0 or S >= 3 else None,
                  seq=torch.tensor(bounds, dtype=torch.int32, device=DEV) if S > 1 else None,
                  d_loss=torch.full((1,), 0.75, device=DEV),
                  d_w=(torch.randn((T, k), generator=_gen(seed, 6), device=DEV) * 1e-3
                       if case["weights"] else None))
    elif op == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        _, _, w, row_idx, _ = _routing(T, case["E"], k, seed)
        st.update(w=w, row_idx=row_idx, d_out=_normal((T, H), 1e-2, _gen(seed, 7)),
                  y=torch.randn((T * k, H), generator=_gen(seed, 8), device=DEV).to(dt))
    elif op == "quantize":
        T, K, k = case["T"], case["K"], case["k"]
        _, _, _, row_idx, offsets = _routing(T, case["E"], k, seed)
        x = _normal((T, K), 1.0, _gen(seed, 9))
        x[:, ::97] *= 12.0                   # outlier channels
        st.update(x=x, row_idx=row_idx, offsets=offsets)
    else:
        n, K, N, G, fmt = case["n"], case["K"], case["N"], case["G"], case["fmt"]
        offsets = _offsets(case, seed)
        rows = 2 * N if op == "swiglu" else N
        a = _plain_quantize(_normal((n, K), 1.0, _gen(seed, 10)), fmt, 0)
        we = 0 if fmt == "mx" else -6        # weights of 0.02: lifts the block scales into e4m3
        wq = torch.empty((G, rows, K // 2), dtype=torch.uint8, device=DEV)
        ws = torch.empty((G * rows, K // BLOCK[fmt]), dtype=torch.uint8, device=DEV)
        gen = _gen(seed, 11)
        for g in range(G):
            q, s = _plain_quantize(_normal((rows, K), 0.02, gen), fmt, we)
            wq[g] = q
            ws[g * rows:(g + 1) * rows] = s
        st.update(offsets=offsets, a_q=a[0], a_sf=_place_scales(a[1], offsets, G), a_exp=0,
                  w_q=wq, w_sf=_place_scales(ws, None, 1), w_exp=we)
    return st


# ------------------------------------------------------------------ 4-bit layout
def scale_rows(n, offsets, G):
    """Rows of the scale layout's 128-row blocks that n rows take."""
    return 128 * ((n + 127) // 128 if offsets is None else n // 128 + G)


def scale_index(n, nb, offsets, G):
    """[n, nb] positions of the scale bytes of rows 0..n-1 (nb blocks each)."""
    r = torch.arange(n, device=DEV)
    if offsets is None:
        blk, rr = r // 128, r % 128
    else:
        off = offsets.to(torch.int64)
        g = torch.searchsorted(off[1:].contiguous(), r, right=True).clamp(max=G - 1)
        local = r - off[g]
        blk, rr = off[g] // 128 + g + local // 128, local % 128
    b = torch.arange(nb, device=DEV)
    return ((blk[:, None] * (nb // 4) + b[None, :] // 4) * 512 +
            ((rr % 32) * 16 + (rr // 32) * 4)[:, None] + (b % 4)[None, :])


def _place_scales(s, offsets, G):
    n, nb = s.shape
    out = torch.zeros(scale_rows(n, offsets, G) * nb, dtype=torch.uint8, device=DEV)
    for i in range(0, n, 65536):
        pos = scale_index(n, nb, offsets, G)[i:i + 65536] if offsets is not None else \
            scale_index(min(65536, n - i), nb, None, 1) + i * nb
        out[pos.reshape(-1)] = s[i:i + 65536].reshape(-1)
    return out


# ------------------------------------------------------------------ plain form
def _e2m1_code(v):
    """Nearest e2m1 magnitude's code (ties to the even code, beyond 6 to 6) and
    the sign bit above it."""
    a = v.abs()
    c = torch.zeros_like(a, dtype=torch.uint8)
    for mid, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                    (3.5, True), (5.0, False)):
        c += (a >= mid) if up else (a > mid)
    return c | (torch.signbit(v).to(torch.uint8) << 3)


def _pow2(e):
    """2^e in fp32 for an integer tensor e in [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _plain_quantize(x, fmt, scale_exp):
    """-> (packed codes [n, K/2], scale bytes [n, K/block])."""
    n, K = x.shape
    f = x.to(torch.float32).view(n, -1, BLOCK[fmt])
    amax = f.abs().amax(2)
    if fmt == "mx":
        _, e = torch.frexp(amax)             # amax = m 2^e, 1/2 <= m < 1
        b = torch.where(amax > 0, e - 1 - 2 + 127, torch.zeros_like(e)).clamp(0, 254)
        v = f * _pow2(127 - b)[:, :, None]
    else:
        s8 = (amax / 6.0 * 2.0 ** -scale_exp).clamp(max=448.0).to(torch.float8_e4m3fn)
        b = s8.view(torch.uint8)
        s = (s8.to(torch.float32) * 2.0 ** scale_exp)[:, :, None]
        v = torch.where(s > 0, f / s, torch.zeros_like(f))
    c = _e2m1_code(v).view(n, K)
    return c[:, 0::2] | (c[:, 1::2] << 4), b.to(torch.uint8)


def _scale_values(b, fmt, scale_exp):
    if fmt == "mx":
        return _pow2(b.to(torch.int32) - 127)
    return b.view(torch.float8_e4m3fn).to(torch.float32) * 2.0 ** scale_exp


def _plain_values(q, s, fmt, scale_exp):
    """fp32 values of packed codes [n, K/2] with scale bytes [n, K/block]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    v = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), 2).view(q.shape[0], -1)
    sv = _scale_values(s, fmt, scale_exp)
    return (v.view(q.shape[0], -1, BLOCK[fmt]) * sv[:, :, None]).view(q.shape[0], -1)


def _plain_router(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    lg, idx = st["logits"], st["idx"].long()
    mask = st["mask"].bool() if st["mask"] is not None else \
        torch.ones(T, dtype=torch.bool, device=DEV)
    seq = st["seq"].long() if st["seq"] is not None else torch.tensor([0, T], device=DEV)
    S = seq.numel() - 1
    sid = torch.searchsorted(seq[1:].contiguous(), torch.arange(T, device=DEV), right=True)
    lg = torch.where(mask[:, None], lg, torch.zeros_like(lg))
    ex = torch.exp(lg - lg.amax(1, keepdim=True))
    p = ex / ex.sum(1, keepdim=True) * mask[:, None]
    n = torch.zeros(S, dtype=torch.int32, device=DEV).index_add_(0, sid, mask.to(torch.int32))
    counts = torch.zeros(S * E, dtype=torch.int32, device=DEV)
    counts.index_add_(0, (sid[:, None] * E + idx).reshape(-1),
                      mask[:, None].expand(T, k).reshape(-1).to(torch.int32))
    counts = counts.view(S, E)
    n1 = n.clamp(min=1).to(torch.float64)
    sums = torch.zeros((S, E), dtype=torch.float64, device=DEV)
    sums.index_add_(0, sid, p.to(torch.float64))
    prob = sums / n1[:, None]
    full = (n > 0).sum().clamp(min=1).to(torch.float64)
    loss = (st["coef"] * E / (k * full) * ((counts * prob).sum(1) / n1).sum()).to(torch.float32)
    scale = (st["d_loss"] * st["coef"] * E / (k * full * n1 * n1)).to(torch.float32)[sid]
    cs = counts.to(torch.float32)[sid]
    d = scale[:, None] * p * (cs - (p * cs).sum(1, keepdim=True))
    if st["d_w"] is not None:
        ps = torch.gather(p, 1, idx)
        dw = st["d_w"]
        if c["renorm"]:
            w = ps / ps.sum(1, keepdim=True).clamp(min=1e-30)
            d.scatter_add_(1, idx, w * (dw - (w * dw).sum(1, keepdim=True)))
        else:
            d = d - p * (ps * dw).sum(1, keepdim=True)
            d.scatter_add_(1, idx, ps * dw)
        d = d * mask[:, None]
    return dict(loss=loss, counts=counts, prob_mean=prob.to(torch.float32), d_logits=d)


def _plain_combine(st):
    T, H, k = st["case"]["T"], st["case"]["H"], st["case"]["k"]
    y, w = st["y"], st["w"]
    d = st["d_out"].to(torch.float32)
    d_y = torch.empty_like(y)
    d_w = torch.empty_like(w)
    rows = st["row_idx"].view(T, k).long()
    for j in range(k):
        d_w[:, j] = (y[rows[:, j]].to(torch.float32) * d).sum(1)
        d_y[rows[:, j]] = (w[:, j:j + 1] * d).to(y.dtype)
    return dict(d_y=d_y, d_w=d_w)


def _plain_fake_quantize(st):
    c = st["case"]
    q, s = _plain_quantize(st["x"], c["fmt"], 0)
    v = _plain_values(q, s, c["fmt"], 0).to(torch.bfloat16)
    out = torch.empty((c["T"] * c["k"], c["K"]), dtype=torch.bfloat16, device=DEV)
    rows = st["row_idx"].view(c["T"], c["k"]).long()
    for j in range(c["k"]):
        out[rows[:, j]] = v
    return out


def _plain_product(st):
    c = st["case"]
    n, K, N, G, fmt = c["n"], c["K"], c["N"], c["G"], c["fmt"]
    nb = K // BLOCK[fmt]
    rows = st["w_q"].shape[1]
    off = st["offsets"].tolist()
    out = torch.empty((n, N), dtype=torch.float32 if c["f32"] else torch.bfloat16, device=DEV)
    pos = scale_index(n, nb, st["offsets"], G)
    wpos = scale_index(rows, nb, None, 1)
    for g in range(G):
        a, b = off[g], off[g + 1]
        if a == b:
            continue
        av = _plain_values(st["a_q"][a:b], st["a_sf"][pos[a:b]], fmt, st["a_exp"])
        wv = _plain_values(st["w_q"][g], st["w_sf"][wpos + g * rows * nb], fmt, st["w_exp"])
        y = av @ wv.T
        if c["op"] == "swiglu":
            gate, up = y[:, :N], y[:, N:]
            y = gate / (1.0 + torch.exp(-gate)) * up
        out[a:b] = y.to(out.dtype)
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return {"router": _plain_router, "combine": _plain_combine,
                "quantize": _plain_fake_quantize, "swiglu": _plain_product,
                "matmul": _plain_product}[op](state)
    import moe_expert_routing_fp32_gb300 as moe
    if op == "router":
        bal = moe.balance_loss(state["logits"], state["idx"], state["coef"],
                               token_mask=state["mask"], seq_offsets=state["seq"])
        d = moe.gate_topk_backward(state["logits"], state["idx"], state["d_w"],
                                   renorm=c["renorm"], balance=bal, d_loss=state["d_loss"],
                                   token_mask=state["mask"], seq_offsets=state["seq"])
        return dict(loss=bal["loss"], counts=bal["counts"], prob_mean=bal["prob_mean"],
                    d_logits=d)
    if op == "combine":
        d_y, d_w = moe.finalize_routing_backward(state["d_out"], state["y"], state["row_idx"],
                                                 state["w"])
        return dict(d_y=d_y, d_w=d_w)
    if op == "quantize":
        m = moe.fp4_quantize(state["x"], c["fmt"], row_idx=state["row_idx"], k=c["k"],
                             offsets=state["offsets"])
        return moe.fp4_dequantize(m, offsets=state["offsets"])
    a = moe.Fp4Matrix(state["a_q"], state["a_sf"], c["fmt"], state["a_exp"])
    w = moe.Fp4Matrix(state["w_q"], state["w_sf"], c["fmt"], state["w_exp"])
    if op == "swiglu":
        return moe.fp4_grouped_swiglu(a, state["offsets"], w)
    return moe.fp4_grouped_matmul(a, state["offsets"], w, out_f32=c["f32"])


# ------------------------------------------------------------------ floors
def work(case):
    op = case["op"]
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        # logits and assignments in, gradients out; the step runs forward then
        # backward, so the logits count once
        b = T * E * 8 + T * k * 4 + (T * k * 4 if case["weights"] else 0) + T
        return {"bytes": b, "flops": T * E * 12}
    if op == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        e = 4 if case["f32"] else 2
        return {"bytes": T * H * 2 + 2 * T * k * H * e + T * k * 12, "flops": 3 * T * k * H}
    if op == "quantize":
        T, K, k = case["T"], case["K"], case["k"]
        return {"bytes": T * K * 2 + T * k * K * 2 + T * k * 4, "flops": 4 * T * K}
    n, K, N = case["n"], case["K"], case["N"]
    rows = 2 * N if op == "swiglu" else N
    per = 0.5 + 1.0 / BLOCK[case["fmt"]]
    return {"bytes": int((n + case["active"] * rows) * K * per) + n * N * (4 if case["f32"] else 2),
            "flops": 2 * n * K * rows}


# ------------------------------------------------------------------ 64 bits
def _exact_grid(x, fmt):
    """The value that each element of x (fp64, blocks in the last dimension)
    is held as: nearest multiple of the grid's step at its magnitude."""
    amax = x.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        # 2^floor(log2 amax): amax over its significand, which lies in [1, 2)
        amax = amax.clamp(min=2.0 ** -200)
        s = (amax / (2.0 * torch.frexp(amax)[0]) / 4.0).clamp(min=2.0 ** -127)
    else:
        t = amax / 6.0
        t1 = t.clamp(min=2.0 ** -6)
        step = t1 / (2.0 * torch.frexp(t1)[0]) / 8.0
        s = (torch.round(t / step) * step).clamp(max=448.0)
    v = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(torch.float64)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=6.0) * s


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


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        seq = [0, T] if st["seq"] is None else st["seq"].tolist()
        d = torch.zeros((T, E), dtype=torch.float64, device=DEV)
        S = len(seq) - 1
        counts = torch.zeros((S, E), dtype=torch.int32, device=DEV)
        prob = torch.zeros((S, E), dtype=torch.float64, device=DEV)
        loss = torch.zeros((), dtype=torch.float64, device=DEV)
        keep = torch.ones(T, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"] != 0
        live = [s for s in range(S) if bool(keep[seq[s]:seq[s + 1]].any())]
        for s in live:
            t = torch.nonzero(keep[seq[s]:seq[s + 1]])[:, 0] + seq[s]
            i = st["idx"][t].long()
            p = torch.softmax(st["logits"][t].to(torch.float64), 1)
            c = torch.bincount(i.reshape(-1), minlength=E)
            counts[s] = c.to(torch.int32)
            c = c.to(torch.float64)
            m = t.numel()
            prob[s] = p.sum(0) / m
            a = st["coef"] * E / (k * m * len(live))
            loss += a * (c * prob[s]).sum()
            gp = 0.75 * a / m * c[None, :].expand(m, E).clone()        # d loss / d p
            if st["d_w"] is not None:
                dw = st["d_w"][t].to(torch.float64)
                sel = torch.gather(p, 1, i)
                if case["renorm"]:
                    z = sel.sum(1, keepdim=True)
                    gp.scatter_add_(1, i, dw / z - (dw * sel).sum(1, keepdim=True) / (z * z))
                else:
                    gp.scatter_add_(1, i, dw)
            d[t] = p * (gp - (p * gp).sum(1, keepdim=True))
        return dict(loss=loss, counts=counts, prob_mean=prob, d_logits=d)
    if op == "combine":
        T, H, k = case["T"], case["H"], case["k"]
        d_y = torch.empty((T * k, H), dtype=torch.float64, device=DEV)
        d_w = torch.empty((T * k,), dtype=torch.float64, device=DEV)
        rows = st["row_idx"].long()
        for a in range(0, T * k, 8192):
            r = rows[a:a + 8192]
            tok = torch.arange(a, a + r.numel(), device=DEV) // k
            g = st["d_out"][tok].to(torch.float64)
            d_w[a:a + 8192] = torch.einsum("nh,nh->n", g, st["y"][r].to(torch.float64))
            d_y[r] = g * st["w"].view(-1)[a:a + 8192, None].to(torch.float64)
        return dict(d_y=d_y, d_w=d_w.view(T, k))
    if op == "quantize":
        T, K, k, fmt = case["T"], case["K"], case["k"], case["fmt"]
        out = torch.empty((T * k, K), dtype=torch.float64, device=DEV)
        rows = st["row_idx"].view(T, k).long()
        for a in range(0, T, 4096):
            x = st["x"][a:a + 4096].to(torch.float64)
            v = _exact_grid(x.view(x.shape[0], -1, BLOCK[fmt]), fmt).view(x.shape)
            for j in range(k):
                out[rows[a:a + 4096, j]] = v
        return out
    n, K, N, G, fmt = case["n"], case["K"], case["N"], case["G"], case["fmt"]
    nb = K // BLOCK[fmt]
    rows = st["w_q"].shape[1]
    off = st["offsets"].tolist()
    out = torch.empty((n, N), dtype=torch.float64, device=DEV)
    for g in range(G):
        a, b = off[g], off[g + 1]
        if b <= a:
            continue
        # the scale tiles as [row block, block of 4, row % 32, row / 32, 4]
        first = a // 128 + g
        m = (b - a + 127) // 128
        t = st["a_sf"].view(-1, nb // 4, 32, 4, 4)[first:first + m]
        sa = t.permute(0, 3, 2, 1, 4).reshape(m * 128, nb)[:b - a]
        t = st["w_sf"].view(-1, nb // 4, 32, 4, 4)[g * rows // 128:(g + 1) * rows // 128]
        sw = t.permute(0, 3, 2, 1, 4).reshape(rows, nb)
        y = _exact_values(st["a_q"][a:b], sa, fmt, st["a_exp"]) @ \
            _exact_values(st["w_q"][g], sw, fmt, st["w_exp"]).T
        out[a:b] = torch.sigmoid(y[:, :N]) * y[:, :N] * y[:, N:] if op == "swiglu" else y
    return out
