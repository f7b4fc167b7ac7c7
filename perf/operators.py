"""The layer operators' cases for measurement: linear attention with a decay
for each head (chunked forward, backward, single-token step), the
root-mean-square norm with the residual's addition (outputs in the inputs' type
or in 8 bits with scales, and its gradients) and the rotary positions of q and k.

``run`` computes a case either in plain torch operations in 32 bits (``own``
false) or through the package's entry points (``own`` true); ``exact`` computes
it in 64 bits from the token recurrence (linear attention) or the row formula.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6
PLAIN_CHUNK = 64        # chunk length of the plain forms of linear attention


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def listed():
    return [
        # prompt of a long-context layer: the repository's longest prefill shape
        dict(name="attn_fwd_t65536_h32", op="attn_fwd", B=1, T=65536, H=32, Hk=32, dk=128, dv=128,
             dtype=BF16, decay="token", resets=False, h0=False),
        # a training batch's forward (the repository's 4 x 4096 x 16 x 128 shape)
        dict(name="attn_fwd_b4_t4096_h16", op="attn_fwd", B=4, T=4096, H=16, Hk=16, dk=128,
             dv=128, dtype=BF16, decay="slow", resets=False, h0=False),
        # packed documents in one ragged row, few heads, keys shared by two heads,
        # continuing from a state: every document's first token clears the state
        dict(name="attn_fwd_packed_t29999_h4", op="attn_fwd", B=1, T=29999, H=4, Hk=2, dk=128,
             dv=128, dtype=BF16, decay="slow", resets=True, h0=True),
        # a small full-precision call with one fixed decay for each head
        dict(name="attn_fwd_f32_t257_h2", op="attn_fwd", B=1, T=257, H=2, Hk=2, dk=64, dv=64,
             dtype=F32, decay="head", resets=False, h0=True),
        # the same training batch's backward
        dict(name="attn_bwd_b4_t4096_h16", op="attn_bwd", B=4, T=4096, H=16, Hk=16, dk=128,
             dv=128, dtype=BF16, decay="slow", resets=False, h0=False),
        # a short ragged backward with shared keys, unequal widths and a state
        dict(name="attn_bwd_b2_t777_h4", op="attn_bwd", B=2, T=777, H=4, Hk=2, dk=64, dv=128,
             dtype=BF16, decay="token", resets=True, h0=True),
        # one decode step of a full batch (the repository's decode shape)
        dict(name="attn_step_n256_h32", op="attn_step", N=256, H=32, Hk=32, dk=128, dv=128,
             dtype=BF16, decay="token"),
        # the norm before a layer's 8-bit projections, over a long prompt
        dict(name="norm_fp8_r65536_d4096", op="norm_fwd", rows=65536, D=4096, dtype=BF16,
             quant=True),
        # the same for a few decoding sequences: latency
        dict(name="norm_fp8_r5_d2048", op="norm_fwd", rows=5, D=2048, dtype=BF16, quant=True),
        # the norm's gradients over a training batch
        dict(name="norm_bwd_r16384_d2048", op="norm_bwd", rows=16384, D=2048, dtype=BF16),
        # rotary positions of a training batch, halves of the head paired
        dict(name="rotary_b4_t4096_h16", op="rotary", B=4, T=4096, H=16, Hk=16, d=128, rot=128,
             dtype=BF16, interleaved=False, inverse=False),
        # one decoding token of each of a few sequences, a quarter of the head,
        # neighbours paired, keys shared by eight heads
        dict(name="rotary_n7_t1_h32", op="rotary", B=7, T=1, H=32, Hk=4, d=128, rot=32,
             dtype=BF16, interleaved=True, inverse=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "attn_step", "norm_fwd",
                     "norm_bwd", "rotary"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    if op in ("attn_fwd", "attn_bwd"):
        # token-heads up to the listed calls' (an eighth of that in full precision)
        most = (2 ** 21 if op == "attn_fwd" else 2 ** 18) // (8 if dtype == F32 else 1)
        H = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
        B = rng.choice([1, 1, 2, 3, 4])
        T = min(_log_int(rng, 1, 65536), max(1, most // (B * H)))
        Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
        decay = rng.choice(["token", "slow", "head"])
        return dict(op=op, B=B, T=T, H=H, Hk=Hk, dk=rng.choice([64, 128]),
                    dv=rng.choice([64, 128]), dtype=dtype, decay=decay,
                    resets=decay != "head" and rng.random() < 0.5, h0=rng.random() < 0.5)
    if op == "attn_step":
        H = rng.choice([1, 2, 4, 8, 16, 32])
        return dict(op=op, N=_log_int(rng, 1, 256), H=H,
                    Hk=rng.choice([h for h in range(1, H + 1) if H % h == 0]),
                    dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), dtype=dtype,
                    decay=rng.choice(["token", "head"]))
    if op == "norm_fwd":
        D = 8 * _log_int(rng, 8, 1024)
        return dict(op=op, rows=min(_log_int(rng, 1, 65536), max(1, 2 ** 28 // D // 2)), D=D,
                    dtype=dtype, quant=rng.random() < 0.6)
    if op == "norm_bwd":
        D = 8 * _log_int(rng, 8, 1024)
        return dict(op=op, rows=min(_log_int(rng, 1, 65536), max(1, 2 ** 25 // D)), D=D,
                    dtype=dtype)
    H = rng.choice([1, 2, 4, 8, 16, 32])
    d = rng.choice([64, 128])
    B = _log_int(rng, 1, 64)
    return dict(op=op, B=B, T=max(1, min(_log_int(rng, 1, 16384), 2 ** 18 // (B * H))), H=H,
                Hk=rng.choice([h for h in range(1, H + 1) if H % h == 0]), d=d,
                rot=rng.choice([d, d, d // 2, d // 4]), dtype=dtype,
                interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5)


# --------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


def _log_decay(gen, case, lead, H):
    """Natural-log decay, [*lead, H] or [H] in 32 bits."""
    if case["decay"] == "head":       # fixed decays 1 - 2^-5 ... 1 - 2^-12 over the heads
        e = torch.linspace(5.0, 12.0, H, device="cuda")
        return torch.log1p(-torch.exp2(-e)) * (1.0 + 0.01 * _randn(gen, H))
    x = _randn(gen, *lead, H)
    if case["decay"] == "slow":       # gates that keep tens to hundreds of tokens
        g = torch.nn.functional.logsigmoid(x + 1.0) / 16.0
    else:                             # strong data-dependent gates
        g = -torch.nn.functional.softplus(x)
    if case.get("resets"):            # about one document in 700 tokens starts anew
        u = torch.rand(*lead, H, generator=gen, device="cuda")[..., :1]
        g = torch.where(u < 1.0 / 700.0, torch.full_like(g, -math.inf), g)
    return g.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], _dtype(case)
    s = {"case": dict(case)}
    if op in ("attn_fwd", "attn_bwd", "attn_step"):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        lead = (case["N"],) if op == "attn_step" else (case["B"], case["T"])
        s["q"] = _unit(_randn(gen, *lead, Hk, dk)).to(dt)
        s["k"] = _unit(_randn(gen, *lead, Hk, dk)).to(dt)
        s["v"] = _randn(gen, *lead, H, dv).to(dt)
        s["g"] = _log_decay(gen, case, lead, H)
        s["scale"] = dk ** -0.5
        if op == "attn_step":
            s["state"] = _randn(gen, case["N"], H, dk, dv)
        else:
            s["h0"] = 0.5 * _randn(gen, case["B"], H, dk, dv) if case["h0"] else None
        if op == "attn_bwd":
            s["do"] = _randn(gen, *lead, H, dv).to(dt)
            s["dhT"] = 0.1 * _randn(gen, case["B"], H, dk, dv) if case["h0"] else None
    elif op in ("norm_fwd", "norm_bwd"):
        rows, D = case["rows"], case["D"]
        s["weight"] = 1.0 + 0.1 * _randn(gen, D)
        if op == "norm_fwd":
            s["x"] = _randn(gen, rows, D).to(dt)
            s["residual"] = (2.0 * _randn(gen, rows, D)).to(dt)
        else:
            s["sum"] = (2.0 * _randn(gen, rows, D)).to(dt)
            s["dy"] = _randn(gen, rows, D).to(dt)
            s["dres"] = _randn(gen, rows, D).to(dt)
    else:
        B, T, H, Hk, d, rot = (case[n] for n in ("B", "T", "H", "Hk", "d", "rot"))
        s["q"] = _randn(gen, B, T, H, d).to(dt)
        s["k"] = _randn(gen, B, T, Hk, d).to(dt)
        length = max(32768, T)
        inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        ang = torch.arange(length, device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        start = torch.randint(0, length - T + 1, (B, 1), generator=gen, device="cuda")
        s["pos"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
    return s


# --------------------------------------------------------------- plain forms

def _segsum(g):
    """[..., n] -> [..., n, n]: entry (r, i) is the sum of g over i+1 .. r for
    i <= r (0 on the diagonal) and -inf above it; summed span by span."""
    n = g.shape[-1]
    below = torch.ones(n, n, dtype=torch.bool, device=g.device).tril(-1)
    x = torch.where(below, g[..., :, None], torch.zeros((), device=g.device, dtype=g.dtype))
    x = torch.cumsum(x, dim=-2)
    keep = torch.ones(n, n, dtype=torch.bool, device=g.device).tril(0)
    return torch.where(keep, x, torch.full((), -math.inf, device=g.device, dtype=g.dtype))


def _heads(x, H):
    """[B, T, Hk, d] -> [B, H, T, d] in 32 bits, each head's own copy of a shared one."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2)


def _plain_attn(q, k, v, g, h0, scale):
    """Chunked linear attention with decay in 32 bits: q, k [B,H,T,dk], v
    [B,H,T,dv], g [B,H,T], h0 [B,H,dk,dv]; returns o [B,H,T,dv] and the end state."""
    B, H, T, dk = q.shape
    dv, C = v.shape[-1], PLAIN_CHUNK
    n = -(-T // C)
    pad = lambda x: torch.nn.functional.pad(x, (0, 0, 0, n * C - T)).view(B, H, n, C, -1)  # noqa: E731
    q, k, v = pad(q), pad(k), pad(v)
    g = torch.nn.functional.pad(g, (0, n * C - T)).view(B, H, n, C)
    decay = torch.exp(_segsum(g))                                   # [B,H,n,C,C]
    inner = (q @ k.transpose(-1, -2) * decay) @ v
    first = torch.exp(torch.cumsum(g, -1))                          # from the chunk's start
    last = decay[..., -1, :]                                        # to the chunk's end
    local = (k * last[..., None]).transpose(-1, -2) @ v             # [B,H,n,dk,dv]
    total = torch.nn.functional.pad(g.sum(-1), (1, 0))              # a chunk "before" the first
    across = torch.exp(_segsum(total))                              # [B,H,n+1,n+1]
    states = torch.cat([h0[:, :, None], local], 2).reshape(B, H, n + 1, dk * dv)
    states = (across @ states).view(B, H, n + 1, dk, dv)
    o = inner + first[..., None] * (q @ states[:, :, :n])
    return scale * o.reshape(B, H, n * C, dv)[:, :, :T], states[:, :, n]


def _gate(g, B, T, H):
    return (g.float().view(1, 1, H).expand(B, T, H) if g.dim() == 1 else g).transpose(1, 2)


def _plain_attn_fwd(s):
    c = s["case"]
    B, T, H = c["B"], c["T"], c["H"]
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(B, H, c["dk"], c["dv"], device="cuda")
    o, hT = _plain_attn(_heads(s["q"], H), _heads(s["k"], H), _heads(s["v"], H),
                        _gate(s["g"], B, T, H), h0, s["scale"])
    return {"o": o.transpose(1, 2).to(s["q"].dtype).contiguous(), "hT": hT}


def _plain_attn_bwd(s):
    c = s["case"]
    B, T, H = c["B"], c["T"], c["H"]
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(B, H, c["dk"], c["dv"], device="cuda")
    leaf = [t.float().detach().requires_grad_() for t in (s["q"], s["k"], s["v"], s["g"], h0)]
    q, k, v, g, h = leaf
    o, hT = _plain_attn(_heads(q, H), _heads(k, H), _heads(v, H), _gate(g, B, T, H), h,
                        s["scale"])
    loss = (o * s["do"].float().transpose(1, 2)).sum()
    if s["dhT"] is not None:
        loss = loss + (hT * s["dhT"]).sum()
    dq, dk, dv, dg, dh = torch.autograd.grad(loss, leaf)
    dt = s["q"].dtype
    return {"q": dq.to(dt), "k": dk.to(dt), "v": dv.to(dt), "g": dg, "h0": dh}


def _plain_attn_step(s):
    H = s["v"].shape[1]
    r = H // s["q"].shape[1]
    q, k = (s[n].float().repeat_interleave(r, dim=1) for n in ("q", "k"))
    a = torch.exp(s["g"])[..., None, None]
    state = s["state"].mul_(a).add_(k[..., :, None] * s["v"].float()[..., None, :])
    o = s["scale"] * (q[..., None, :] @ state)[..., 0, :]
    return {"o": o.to(s["q"].dtype), "state": state}


def _blocks(y):
    """Largest magnitude of each 128-column block of each row, and the padded view."""
    rows, D = y.shape
    nb = -(-D // 128)
    yb = torch.nn.functional.pad(y, (0, nb * 128 - D)).view(rows, nb, 128)
    amax = yb.abs().amax(-1)
    return yb, torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))


def _plain_norm_fwd(s):
    dt, D = s["x"].dtype, s["x"].shape[1]
    r = (s["x"].float() + s["residual"].float()).to(dt)
    x = r.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"]
    if not s["case"]["quant"]:
        return {"y": y.to(dt), "residual": r}
    yb, scale = _blocks(y)
    y8 = (yb / scale[..., None]).reshape(y.shape[0], -1)[:, :D].to(torch.float8_e4m3fn)
    return {"y": y8, "scale": scale, "residual": r}


def _plain_norm_bwd(s):
    dt, D = s["sum"].dtype, s["sum"].shape[1]
    x, dy = s["sum"].float(), s["dy"].float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    wd = dy * s["weight"]
    dx = inv * (wd - x * (inv * inv) * ((wd * x).sum(-1, keepdim=True) / D)) + s["dres"].float()
    return {"x": dx.to(dt), "weight": (dy * x * inv).sum(0)}


def _turn(x, cos, sin, rot, interleaved):
    head, tail = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, tail], -1)


def _plain_rotary(s, up=torch.float32):
    c = s["case"]
    pos = s["pos"].long()
    cos, sin = s["cos"][pos][:, :, None].to(up), s["sin"][pos][:, :, None].to(up)
    if c["inverse"]:
        sin = -sin
    return {n: _turn(s[n].to(up), cos, sin, c["rot"], c["interleaved"]) for n in ("q", "k")}


# --------------------------------------------------------------- the calls

def _own(s):
    import gated_delta_rule_10_gb300 as gdr
    c = s["case"]
    op = c["op"]
    if op == "attn_fwd":
        o, hT = gdr.decay_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], scale=s["scale"])
        return {"o": o, "hT": hT}
    if op == "attn_bwd":
        return gdr.decay_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["h0"], s["dhT"],
                                   scale=s["scale"])
    if op == "attn_step":
        o = gdr.decay_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    if op == "norm_fwd":
        if c["quant"]:
            y, scale, r = gdr.add_rmsnorm_fp8(s["x"], s["residual"], s["weight"], EPS)
            return {"y": y, "scale": scale, "residual": r}
        y, r = gdr.add_rmsnorm(s["x"], s["residual"], s["weight"], EPS)
        return {"y": y, "residual": r}
    if op == "norm_bwd":
        dx, dw = gdr.add_rmsnorm_bwd(s["dy"], s["sum"], s["weight"], EPS, dres=s["dres"])
        return {"x": dx, "weight": dw}
    q, k = gdr.rotary(s["q"], s["k"], s["cos"], s["sin"], s["pos"],
                      interleaved=c["interleaved"], inverse=c["inverse"])
    return {"q": q, "k": k}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rotary":
        return {n: x.to(state[n].dtype) for n, x in _plain_rotary(state).items()}
    return {"attn_fwd": _plain_attn_fwd, "attn_bwd": _plain_attn_bwd,
            "attn_step": _plain_attn_step, "norm_fwd": _plain_norm_fwd,
            "norm_bwd": _plain_norm_bwd}[op](state)


def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == BF16 else 4
    if op in ("attn_fwd", "attn_bwd", "attn_step"):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        if op == "attn_step":
            n, st = case["N"], 2 * case["N"] * H * dk * dv * 4
        else:
            n = case["B"] * case["T"]
            st = (2 if case["h0"] else 1) * case["B"] * H * dk * dv * 4
        gate = 4 * (H if case["decay"] == "head" else n * H)
        io = n * (2 * Hk * dk + 2 * H * dv) * e              # q, k, v read; o written
        flops = 4 * n * H * dk * dv                          # one state update, one read-out
        if op == "attn_bwd":                                 # q, k, v, do read; dq, dk, dv written
            io, gate, flops = n * (4 * Hk * dk + 3 * H * dv) * e, 2 * gate, 10 * n * H * dk * dv
            st = (3 if case["h0"] else 1) * case["B"] * H * dk * dv * 4
        return {"bytes": io + gate + st, "flops": flops}
    if op == "norm_fwd":
        n, D = case["rows"], case["D"]
        y = n * D + 4 * n * -(-D // 128) if case["quant"] else n * D * e
        return {"bytes": 3 * n * D * e + y + 4 * D, "flops": 6 * n * D}
    if op == "norm_bwd":
        n, D = case["rows"], case["D"]
        return {"bytes": 4 * n * D * e + 8 * D, "flops": 10 * n * D}
    n = case["B"] * case["T"]
    return {"bytes": n * (2 * (case["H"] + case["Hk"]) * case["d"] * e + 4 * case["rot"] + 4),
            "flops": 3 * n * (case["H"] + case["Hk"]) * case["rot"]}


# --------------------------------------------------------------- 64 bits

def _exact_attn(s):
    """The token recurrence in 64 bits; with a cotangent also its gradients,
    from the forward states on the way up and their adjoints on the way down."""
    c = s["case"]
    B, T, H, Hk, dk, dv = (c[n] for n in ("B", "T", "H", "Hk", "dk", "dv"))
    r, scale = H // Hk, s["scale"]
    d = lambda n: s[n].double()  # noqa: E731
    q, k, v = d("q").repeat_interleave(r, 2), d("k").repeat_interleave(r, 2), d("v")
    alpha = torch.exp(d("g").expand(B, T, H) if s["g"].dim() == 1 else d("g"))
    S = d("h0").clone() if s["h0"] is not None else torch.zeros(B, H, dk, dv, device="cuda",
                                                               dtype=torch.float64)
    back = "do" in s
    out = torch.empty(B, T, H, dk if back else dv, device="cuda", dtype=torch.float64)
    do = d("do") if back else None
    for t in range(T):
        S.mul_(alpha[:, t, :, None, None])
        S.add_(k[:, t, :, :, None] * v[:, t, :, None, :])
        if back:
            out[:, t] = (S @ do[:, t, :, :, None])[..., 0]
        else:
            out[:, t] = (q[:, t, :, None, :] @ S)[..., 0, :]
    if not back:
        return {"o": scale * out, "hT": S}
    dq = scale * out
    D = d("dhT").clone() if s["dhT"] is not None else torch.zeros_like(S)
    end = (S * D).sum((-1, -2))                                 # <hT, dhT>
    dkk, dvv = torch.empty_like(k), torch.empty_like(v)
    for t in range(T - 1, -1, -1):
        D.add_(scale * q[:, t, :, :, None] * do[:, t, :, None, :])
        dkk[:, t] = (D @ v[:, t, :, :, None])[..., 0]
        dvv[:, t] = (k[:, t, :, None, :] @ D)[..., 0, :]
        D.mul_(alpha[:, t, :, None, None])
    flow = (q * dq).sum(-1) - (k * dkk).sum(-1)                 # by token and head
    dg = flow.flip(1).cumsum(1).flip(1) + end[:, None]
    dg = torch.where(alpha > 0, dg, torch.zeros_like(dg))
    shared = lambda x: x.view(B, T, Hk, r, dk).sum(3)  # noqa: E731
    if s["g"].dim() == 1:
        dg = dg.sum((0, 1))
    return {"q": shared(dq), "k": shared(dkk), "v": dvv, "g": dg, "h0": D}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attn_fwd", "attn_bwd"):
        return _exact_attn(s)
    if op == "attn_step":
        r = case["H"] // case["Hk"]
        q, k = (s[n].double().repeat_interleave(r, 1) for n in ("q", "k"))
        S = s["state"].double() * torch.exp(s["g"].double())[..., None, None]
        S = S + torch.einsum("nhi,nhj->nhij", k, s["v"].double())
        return {"o": s["scale"] * torch.einsum("nhi,nhij->nhj", q, S), "state": S}
    if op == "norm_fwd":
        # the residual is stored in the inputs' type and the norm reads it from there
        r = s["x"].double() + s["residual"].double()
        x = (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()
        y = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS) * s["weight"].double()
        if not case["quant"]:
            return {"y": y, "residual": r}
        D, rows = case["D"], case["rows"]
        wide = torch.zeros(rows, -(-D // 128) * 128, device="cuda", dtype=torch.float64)
        wide[:, :D] = y
        scale = wide.view(rows, -1, 128).abs().amax(-1) / 448.0
        scale[scale == 0] = 1.0
        # the 8-bit values before their last rounding
        return {"y": y / scale.repeat_interleave(128, 1)[:, :D], "scale": scale, "residual": r}
    if op == "norm_bwd":
        x, dy, w = s["sum"].double(), s["dy"].double(), s["weight"].double()
        rms = torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS)
        n = x / rms
        dn = dy * w
        dx = (dn - n * (dn * n).mean(-1, keepdim=True)) / rms
        return {"x": dx + s["dres"].double(), "weight": torch.einsum("rd,rd->d", dy, n)}
    pos = s["pos"].long()
    z = torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, :, None]
    if case["inverse"]:
        z = z.conj()
    out, rot = {}, case["rot"]
    for n in ("q", "k"):
        x = s[n].double().clone()
        if case["interleaved"]:
            y = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2)) * z
            x[..., :rot] = torch.view_as_real(y).flatten(-2)
        else:
            y = torch.complex(x[..., :rot // 2].contiguous(),
                              x[..., rot // 2:rot].contiguous()) * z
            x[..., :rot // 2], x[..., rot // 2:rot] = y.real, y.imag
        out[n] = x
    return out
