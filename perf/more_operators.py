"""The block operators' cases for measurement: the short causal convolution
(prompts, gradients, single tokens), the state space recurrence whose decay
depends on token, channel and state (the same three) and the norms after and
before a block with its gate and residual scale (forward and gradients).

``run`` computes a case either in plain torch operations in 32 bits (``own``
false) or through the package's entry points (``own`` true); ``exact`` computes
it in 64 bits from the token recurrence or the row formula.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def listed():
    return [
        # the convolution over a long prompt, its input one half of a fused projection
        dict(name="conv_fwd_t65536_d4096", op="conv_fwd", B=1, T=65536, D=4096, K=4, dtype=BF16,
             starts=False, state=False, fused=True),
        # its gradients over a training batch of packed documents
        dict(name="conv_bwd_b4_t4096_d4096", op="conv_bwd", B=4, T=4096, D=4096, K=4, dtype=BF16,
             starts=True, state=False, fused=False),
        # one token of each sequence of a full decoding batch: latency
        dict(name="conv_step_n256_d4096", op="conv_step", N=256, D=4096, K=4, dtype=BF16),
        # the recurrence over a long prompt, one sequence
        dict(name="scan_fwd_t65536_d2048", op="scan_fwd", B=1, T=65536, D=2048, G=1, N=16,
             dtype=BF16, z=True, starts=False, h0=False, fused=True),
        # a training batch's forward, documents packed into rows
        dict(name="scan_fwd_b4_t4096_d4096", op="scan_fwd", B=4, T=4096, D=4096, G=1, N=16,
             dtype=BF16, z=True, starts=True, h0=False, fused=False),
        # a small full-precision continuation, three groups of channels
        dict(name="scan_fwd_f32_b2_t257_d192", op="scan_fwd", B=2, T=257, D=192, G=3, N=8,
             dtype=F32, z=False, starts=False, h0=True, fused=False),
        # a training batch's gradients
        dict(name="scan_bwd_b4_t4096_d2048", op="scan_bwd", B=4, T=4096, D=2048, G=1, N=16,
             dtype=BF16, z=True, starts=False, h0=False, fused=False),
        # a short ragged backward from a state, wide states, two groups, packed
        dict(name="scan_bwd_b2_t777_d320", op="scan_bwd", B=2, T=777, D=320, G=2, N=64,
             dtype=BF16, z=False, starts=True, h0=True, fused=False),
        # one decode step of a full batch
        dict(name="scan_step_n256_d4096", op="scan_step", N=256, D=4096, G=1, N_state=16,
             dtype=BF16, z=True),
        # norms between two blocks of a long prompt
        dict(name="norms_fwd_r65536_d4096", op="norms_fwd", rows=65536, D=4096, dtype=BF16,
             gate=True, scale=True),
        # the same for a few decoding sequences: latency
        dict(name="norms_fwd_r5_d2048", op="norms_fwd", rows=5, D=2048, dtype=BF16, gate=True,
             scale=True),
        # their gradients over a training batch
        dict(name="norms_bwd_r16384_d2048", op="norms_bwd", rows=16384, D=2048, dtype=BF16,
             gate=True, scale=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd",
                     "scan_bwd", "scan_step", "norms_fwd", "norms_bwd"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    wide = 2 if dtype == F32 else 1
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("conv_fwd", "conv_bwd"):
        D = 8 * _log_int(rng, 1, 1024)
        B = rng.choice([1, 1, 2, 3, 4])
        most = 2 ** (28 if op == "conv_fwd" else 26) // wide
        return dict(op=op, B=B, T=max(1, min(_log_int(rng, 1, 65536), most // (B * D))), D=D,
                    K=rng.choice([2, 3, 4, 4]), dtype=dtype, starts=flag(), state=flag(),
                    fused=flag())
    if op == "conv_step":
        return dict(op=op, N=_log_int(rng, 1, 256), D=8 * _log_int(rng, 8, 512),
                    K=rng.choice([2, 3, 4, 4]), dtype=dtype)
    if op in ("scan_fwd", "scan_bwd"):
        N, G, B = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 3]), rng.choice([1, 1, 2, 4])
        D = 8 * G * _log_int(rng, 1, 512 // G)
        most = 2 ** (31 if op == "scan_fwd" else 29) // wide
        return dict(op=op, B=B, T=max(1, min(_log_int(rng, 1, 65536 if op == "scan_fwd" else 8192),
                                             most // (B * D * N))),
                    D=D, G=G, N=N, dtype=dtype, z=flag(), starts=flag(), h0=flag(), fused=flag())
    if op == "scan_step":
        G = rng.choice([1, 1, 2, 3])
        return dict(op=op, N=_log_int(rng, 1, 256), D=8 * G * _log_int(rng, 4, 512 // G), G=G,
                    N_state=rng.choice([8, 16]), dtype=dtype, z=flag())
    D = 8 * _log_int(rng, 8, 1024)
    most = 2 ** (27 if op == "norms_fwd" else 25) // wide
    return dict(op=op, rows=min(_log_int(rng, 1, 65536), max(1, most // D)), D=D, dtype=dtype,
                gate=flag(), scale=flag())


# --------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _starts(gen, B, T):
    """True at a document's first token, one in about 700."""
    return torch.rand(B, T, generator=gen, device="cuda") < 1.0 / 700.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], _dtype(case)
    s = {"case": dict(case)}
    if op.startswith("conv"):
        D, K = case["D"], case["K"]
        s["weight"] = _randn(gen, D, K) * K ** -0.5
        s["bias"] = 0.1 * _randn(gen, D)
        if op == "conv_step":
            s["x"] = _randn(gen, case["N"], D).to(dt)
            s["state"] = _randn(gen, case["N"], K - 1, D).to(dt)
            return s
        B, T = case["B"], case["T"]
        if case["fused"]:      # the first part of a projection of twice the width
            s["x"] = torch.randn(B, T, 2 * D, generator=gen, device="cuda", dtype=dt)[..., :D]
        else:
            s["x"] = _randn(gen, B, T, D).to(dt)
        s["starts"] = _starts(gen, B, T) if case["starts"] else None
        s["state"] = _randn(gen, B, K - 1, D).to(dt) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = _randn(gen, B, T, D).to(dt)
            s["dstate"] = _randn(gen, B, K - 1, D).to(dt) if case["state"] else None
    elif op.startswith("scan"):
        D, G = case["D"], case["G"]
        step = op == "scan_step"
        N, lead = (case["N_state"], (case["N"],)) if step else (case["N"], (case["B"], case["T"]))
        # rates -1 ... -N and steps from 0.001 to 0.1 by channel, as layers start out
        s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * _randn(gen, D, N))
        size = torch.exp(torch.rand(D, generator=gen, device="cuda") * math.log(100.0)) * 1e-3
        s["dt_bias"] = torch.log(torch.expm1(size))
        s["dt"] = (0.5 * _randn(gen, *lead, D)).to(dt)
        s["skip"] = 1.0 + 0.1 * _randn(gen, D)
        s["x"] = torch.nn.functional.silu(_randn(gen, *lead, D)).to(dt)
        if not step and case["fused"]:     # parts of the projections that make them
            zx = torch.randn(*lead, 2 * D, generator=gen, device="cuda", dtype=dt)
            s["z"] = zx[..., D:] if case["z"] else None
            p = torch.randn(*lead, 64 + 2 * G * N, generator=gen, device="cuda", dtype=dt)
            s["B"] = p[..., 64:64 + G * N].unflatten(-1, (G, N))
            s["C"] = p[..., 64 + G * N:].unflatten(-1, (G, N))
        else:
            s["z"] = _randn(gen, *lead, D).to(dt) if case["z"] else None
            s["B"] = _randn(gen, *lead, G, N).to(dt)
            s["C"] = _randn(gen, *lead, G, N).to(dt)
        if step:
            s["state"] = _randn(gen, case["N"], D, N)
            return s
        B, T = lead
        s["starts"] = _starts(gen, B, T) if case["starts"] else None
        s["h0"] = _randn(gen, B, D, N) if case["h0"] else None
        if op == "scan_bwd":
            s["dy"] = _randn(gen, B, T, D).to(dt)
            s["dhT"] = 0.1 * _randn(gen, B, D, N) if case["h0"] else None
    else:
        rows, D = case["rows"], case["D"]
        s["post"] = 1.0 + 0.1 * _randn(gen, D)
        s["pre"] = 1.0 + 0.1 * _randn(gen, D)
        s["gate"] = torch.randn(rows, D, generator=gen, device="cuda", dtype=dt) if case["gate"] \
            else None
        s["scale"] = 0.5 + 0.1 * _randn(gen, D) if case["scale"] else None
        s["x"] = torch.randn(rows, D, generator=gen, device="cuda", dtype=dt)
        s["residual"] = 2.0 * torch.randn(rows, D, generator=gen, device="cuda", dtype=dt)
        if op == "norms_bwd":
            s["sum"] = _plain_norms_sum(s)
            del s["residual"]
            s["dy"] = _randn(gen, rows, D).to(dt)
            s["dres"] = _randn(gen, rows, D).to(dt)
    return s


# --------------------------------------------------------------- plain forms

def _silu(x):
    return x * torch.sigmoid(x)


def _plain_conv(x, weight, bias, starts, state):
    """x [B,T,D], state [B,K-1,D] in 32 bits: the sums before the activation, and the
    rows that a next call continues from."""
    B, T, D = x.shape
    K = weight.shape[1]
    rows = torch.cat([state if state is not None else x.new_zeros(B, K - 1, D), x], 1)
    doc = None
    if starts is not None:                 # which document a row is of
        doc = torch.nn.functional.pad(starts.int().cumsum(1), (K - 1, 0))
    out = bias.expand(B, T, D)
    for k in range(K):
        tap = rows[:, k:k + T]
        if doc is not None:
            same = doc[:, k:k + T] == doc[:, K - 1:]
            tap = torch.where(same[..., None], tap, torch.zeros((), device=x.device))
        out = out + weight[:, k] * tap
    last = rows[:, T:]
    if doc is not None:
        last = torch.where((doc[:, T:] == doc[:, -1:])[..., None], last,
                           torch.zeros((), device=x.device))
    return out, last


def _plain_conv_fwd(s):
    dt = s["x"].dtype
    state = None if s["state"] is None else s["state"].float()
    out, last = _plain_conv(s["x"].float(), s["weight"], s["bias"], s["starts"], state)
    return {"y": _silu(out).to(dt), "state": last.to(dt)}


def _plain_conv_bwd(s):
    dt = s["x"].dtype
    c = s["case"]
    start = s["state"] if s["state"] is not None else \
        torch.zeros(c["B"], c["K"] - 1, c["D"], device="cuda")
    leaf = [t.float().detach().requires_grad_() for t in (s["x"], s["weight"], s["bias"], start)]
    out, last = _plain_conv(leaf[0], leaf[1], leaf[2], s["starts"], leaf[3])
    loss = (_silu(out) * s["dy"].float()).sum()
    if s["dstate"] is not None:
        loss = loss + (last * s["dstate"].float()).sum()
    dx, dw, db, ds = torch.autograd.grad(loss, leaf)
    return {"x": dx.to(dt), "weight": dw, "bias": db, "state": ds.to(dt)}


def _plain_conv_step(s):
    K = s["weight"].shape[1]
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    out = s["bias"].expand(s["x"].shape)
    for k in range(K):
        out = out + s["weight"][:, k] * rows[:, k].float()
    s["state"].copy_(rows[:, 1:])
    return {"y": _silu(out).to(s["x"].dtype), "state": s["state"]}


def _plain_scan(x, dt, A, Bm, Cm, skip, z, dt_bias, starts, h0):
    """Pieces of about sqrt(T) tokens side by side, each walked token by token: once for
    the pieces' own end states, once more from the states that these chain up to."""
    B, T, D = x.shape
    G, N = Bm.shape[2:]
    P = 1 << max(0, round(math.log2(T) / 2))
    n = -(-T // P)
    delta = torch.nn.functional.softplus(dt + dt_bias)
    keep = torch.ones(B, T, device=x.device) if starts is None else (~starts).float()
    pad = lambda t: torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, n * P - T)) \
        .unflatten(1, (n, P))  # noqa: E731
    u, xx, kk, bb, cc = pad(delta), pad(x), pad(keep), pad(Bm), pad(Cm)
    kk = kk + pad(torch.ones_like(keep)).eq(0)          # behind the end: nothing changes

    def wide(t):                                        # [B,n,G,N] -> by channel
        return t[..., :, None, :].expand(B, n, G, D // G, N).reshape(B, n, D, N)

    def walk(h, P_end=None):
        ys = []
        for j in range(P):
            d = u[:, :, j, :, None]
            a = torch.exp(d * A) * kk[:, :, j, None, None]
            h = a * h + d * xx[:, :, j, :, None] * wide(bb[:, :, j])
            if P_end is None:
                ys.append((h * wide(cc[:, :, j])).sum(-1))
            else:
                P_end = P_end * a
        return (h, P_end) if P_end is not None else (h, torch.stack(ys, 2))

    zero = torch.zeros(B, n, D, N, device=x.device)
    ends, across = walk(zero, torch.ones_like(zero))
    first = [h0 if h0 is not None else zero[:, 0]]
    for i in range(n):
        first.append(across[:, i] * first[-1] + ends[:, i])
    _, y = walk(torch.stack(first[:n], 1))
    y = y.reshape(B, n * P, D)[:, :T] + skip * x
    return (y if z is None else y * _silu(z)), first[n]


def _plain_scan_fwd(s):
    f = lambda n: None if s[n] is None else s[n].float()  # noqa: E731
    y, hT = _plain_scan(f("x"), f("dt"), s["A"], f("B"), f("C"), s["skip"], f("z"), s["dt_bias"],
                        s["starts"], s["h0"])
    return {"y": y.to(s["x"].dtype), "h": hT}


def _plain_scan_bwd(s):
    c = s["case"]
    dt = s["x"].dtype
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(c["B"], c["D"], c["N"], device="cuda")
    names = ["x", "dt", "A", "B", "C", "skip", "dt_bias", "h0"] + (["z"] if c["z"] else [])
    leaf = {n: (h0 if n == "h0" else s[n]).float().detach().requires_grad_() for n in names}
    y, hT = _plain_scan(leaf["x"], leaf["dt"], leaf["A"], leaf["B"], leaf["C"], leaf["skip"],
                        leaf.get("z"), leaf["dt_bias"], s["starts"], leaf["h0"])
    loss = (y * s["dy"].float()).sum()
    if s["dhT"] is not None:
        loss = loss + (hT * s["dhT"]).sum()
    grads = dict(zip(names, torch.autograd.grad(loss, [leaf[n] for n in names])))
    return {n: g.to(dt) if n in ("x", "dt", "B", "C", "z") else g for n, g in grads.items()}


def _plain_scan_step(s):
    G = s["B"].shape[1]
    x = s["x"].float()
    delta = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])
    b, c = (s[n].float().repeat_interleave(x.shape[1] // G, 1) for n in ("B", "C"))
    state = s["state"].mul_(torch.exp(delta[..., None] * s["A"])).add_((delta * x)[..., None] * b)
    y = (state * c).sum(-1) + s["skip"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return {"y": y.to(s["x"].dtype), "state": state}


def _rms(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norms_sum(s):
    x = s["x"].float()
    u = x * _rms(x) * s["post"]
    if s["scale"] is not None:
        u = u * s["scale"]
    if s["gate"] is not None:
        u = u * torch.sigmoid(s["gate"].float())
    return (s["residual"].float() + u).to(s["x"].dtype)


def _plain_norms_fwd(s):
    r = _plain_norms_sum(s)
    f = r.float()
    return {"y": (f * _rms(f) * s["pre"]).to(r.dtype), "residual": r}


def _plain_norms_bwd(s):
    dt, D = s["x"].dtype, s["x"].shape[1]

    def norm_bwd(g, x, w):
        inv = _rms(x)
        g = g * w
        return inv * (g - x * (inv * inv) * ((g * x).sum(-1, keepdim=True) / D))

    x, r, dy = s["x"].float(), s["sum"].float(), s["dy"].float()
    out = {"pre": (dy * r * _rms(r)).sum(0)}
    dr = s["dres"].float() + norm_bwd(dy, r, s["pre"])
    out["residual"] = dr.to(dt)
    unit = x * _rms(x)
    gate = torch.ones((), device="cuda")
    if s["gate"] is not None:
        gate = torch.sigmoid(s["gate"].float())
    scale = s["scale"] if s["scale"] is not None else torch.ones((), device="cuda")
    sums = (dr * gate * unit).sum(0)
    out["post"] = sums * scale
    if s["scale"] is not None:
        out["scale"] = sums * s["post"]
    if s["gate"] is not None:
        out["gate"] = (dr * scale * unit * s["post"] * gate * (1.0 - gate)).to(dt)
    out["x"] = norm_bwd(dr * scale * gate, x, s["post"]).to(dt)
    return out


# --------------------------------------------------------------- the calls

def _own(s):
    import gated_delta_rule_10_gb300 as gdr
    c = s["case"]
    op = c["op"]
    if op == "conv_fwd":
        y, state = gdr.short_conv_fwd(s["x"], s["weight"], s["bias"], s["state"],
                                      starts=s["starts"])
        return {"y": y, "state": state}
    if op == "conv_bwd":
        return gdr.short_conv_bwd(s["dy"], s["x"], s["weight"], s["bias"], s["state"], s["dstate"],
                                  starts=s["starts"])
    if op == "conv_step":
        y = gdr.short_conv_step(s["x"], s["weight"], s["bias"], s["state"])
        return {"y": y, "state": s["state"]}
    if op == "scan_fwd":
        y, hT = gdr.state_space_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h0"],
                                    skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"],
                                    starts=s["starts"])
        return {"y": y, "h": hT}
    if op == "scan_bwd":
        g = gdr.state_space_bwd(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["h0"],
                                s["dhT"], skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"],
                                starts=s["starts"])
        names = ["x", "dt", "A", "B", "C", "skip", "dt_bias", "h0"] + (["z"] if c["z"] else [])
        return {n: g[n] for n in names}
    if op == "scan_step":
        y = gdr.state_space_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"],
                                 skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"])
        return {"y": y, "state": s["state"]}
    if op == "norms_fwd":
        y, r = gdr.block_norms(s["x"], s["residual"], s["post"], s["pre"], EPS, gate=s["gate"],
                               scale=s["scale"])
        return {"y": y, "residual": r}
    g = gdr.block_norms_bwd(s["dy"], s["x"], s["sum"], s["post"], s["pre"], EPS, gate=s["gate"],
                            scale=s["scale"], dres=s["dres"])
    names = ["pre", "residual", "post"] + (["scale"] if c["scale"] else []) + \
        (["gate"] if c["gate"] else []) + ["x"]
    return {n: g[n] for n in names}


def run(state):
    if own:
        return _own(state)
    return {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd,
            "conv_step": _plain_conv_step, "scan_fwd": _plain_scan_fwd,
            "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
            "norms_fwd": _plain_norms_fwd, "norms_bwd": _plain_norms_bwd}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == BF16 else 4
    D = case["D"]
    if op.startswith("conv"):
        K = case["K"]
        if op == "conv_step":          # x and the state read, y and the state written
            return {"bytes": case["N"] * D * e * 2 * K + 4 * D * (K + 1),
                    "flops": 2 * K * case["N"] * D}
        n, edge = case["B"] * case["T"] * D, case["B"] * (K - 1) * D * e
        mask = case["B"] * case["T"] if case["starts"] else 0
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + (2 if case["state"] else 1) * edge + 4 * D * (K + 1) + mask,
                    "flops": (2 * K + 4) * n}
        return {"bytes": 3 * n * e + (3 if case["state"] else 1) * edge + 8 * D * (K + 1) + mask,
                "flops": (6 * K + 8) * n}
    if op.startswith("scan"):
        G = case["G"]
        if op == "scan_step":
            n, N = case["N"], case["N_state"]
            io = n * ((4 if case["z"] else 3) * D + 2 * G * N) * e
            return {"bytes": io + 8 * n * D * N + 4 * D * (N + 2), "flops": 8 * n * D * N}
        n, N = case["B"] * case["T"], case["N"]
        mask = n if case["starts"] else 0
        state = 4 * case["B"] * D * N
        if op == "scan_fwd":           # per token, channel and state: exp, three products, two sums
            io = n * ((4 if case["z"] else 3) * D + 2 * G * N) * e
            return {"bytes": io + mask + (2 if case["h0"] else 1) * state + 4 * D * (N + 2),
                    "flops": 7 * n * D * N}
        io = n * ((7 if case["z"] else 5) * D + 4 * G * N) * e
        return {"bytes": io + mask + (3 if case["h0"] else 1) * state + 8 * D * (N + 2),
                "flops": 22 * n * D * N}
    n = case["rows"] * D * e
    g, sc = int(case["gate"]), int(case["scale"])
    if op == "norms_fwd":              # x, residual, gate read; the sum and y written
        return {"bytes": (4 + g) * n + 4 * D * (2 + sc), "flops": 14 * case["rows"] * D}
    # dy, dres, x, sum, gate read; dx, dresidual, dgate written
    return {"bytes": (6 + 2 * g) * n + 8 * D * (2 + sc), "flops": 34 * case["rows"] * D}


# --------------------------------------------------------------- 64 bits

def _act64(x):
    return x / (1.0 + torch.exp(-x))


def _act64_slope(x):
    sig = 1.0 / (1.0 + torch.exp(-x))
    return sig * (1.0 + x * (1.0 - sig))


def _exact_conv(case, s):
    """Tap by tap: the input j tokens back counts where no document starts in between."""
    K, D = case["K"], case["D"]
    w = s["weight"].double()
    if case["op"] == "conv_step":
        rows = torch.cat([s["state"], s["x"][:, None]], 1).double()
        return {"y": _act64(torch.einsum("nkd,dk->nd", rows, w) + s["bias"].double()),
                "state": rows[:, 1:]}
    B, T = case["B"], case["T"]
    x = s["x"].double()
    begun = s["starts"] if s["starts"] is not None else torch.zeros(B, T, dtype=torch.bool,
                                                                    device="cuda")
    old = s["state"].double() if s["state"] is not None else torch.zeros(B, K - 1, D, device="cuda",
                                                                         dtype=torch.float64)
    # alone[j][b, t]: the tap j tokens back is of another document
    alone, cut = [], torch.zeros(B, T, dtype=torch.bool, device="cuda")
    for j in range(K):
        alone.append(cut.clone())
        if j < T:
            cut = cut.clone()
            cut[:, j:] |= begun[:, :T - j]

    def back(j):
        out = torch.zeros(B, T, D, device="cuda", dtype=torch.float64)
        if j < T:
            out[:, j:] = x[:, :T - j]
        m = min(j, T)
        out[:, :m] = old[:, K - 1 - j:K - 1 - j + m]
        out[alone[j]] = 0.0
        return out

    pre = s["bias"].double() + sum(back(j) * w[:, K - 1 - j] for j in range(K))
    if case["op"] == "conv_fwd":
        state = torch.zeros(B, K - 1, D, device="cuda", dtype=torch.float64)
        for b in range(B):
            for i in range(K - 1):
                t = T - (K - 1) + i
                if not bool(begun[b, max(t + 1, 0):].any()):
                    state[b, i] = x[b, t] if t >= 0 else old[b, T + i]
        return {"y": _act64(pre), "state": state}
    ds = s["dy"].double() * _act64_slope(pre)
    dx, dold = torch.zeros_like(x), torch.zeros_like(old)
    dw = torch.zeros_like(w)
    for j in range(K):
        dw[:, K - 1 - j] = (ds * back(j)).sum((0, 1))
        part = ds * w[:, K - 1 - j]
        part[alone[j]] = 0.0
        if j < T:
            dx[:, :T - j] += part[:, j:]
        m = min(j, T)
        dold[:, K - 1 - j:K - 1 - j + m] += part[:, :m]
    if s["dstate"] is not None:
        for b in range(B):
            for i in range(K - 1):
                t = T - (K - 1) + i
                if not bool(begun[b, max(t + 1, 0):].any()):
                    if t >= 0:
                        dx[b, t] += s["dstate"][b, i].double()
                    else:
                        dold[b, T + i] += s["dstate"][b, i].double()
    return {"x": dx, "weight": dw, "bias": ds.sum((0, 1)), "state": dold}


def _exact_scan(case, s):
    """Token by token, and back with the states kept."""
    step = case["op"] == "scan_step"
    G, D = case["G"], case["D"]
    N = case["N_state"] if step else case["N"]
    d64 = lambda n: s[n].double()  # noqa: E731
    A, skip = d64("A"), d64("skip")
    raw = d64("dt") + d64("dt_bias")
    u = torch.where(raw > 30.0, raw + torch.log1p(torch.exp(-raw.clamp_min(30.0))),
                    torch.log1p(torch.exp(raw.clamp_max(30.0))))
    if step:
        x = d64("x")
        b, c = (d64(n).repeat_interleave(D // G, 1) for n in ("B", "C"))
        h = torch.exp(u[..., None] * A) * d64("state") + (u * x)[..., None] * b
        y = (c * h).sum(-1) + skip * x
        return {"y": y if s["z"] is None else y * _act64(d64("z")), "state": h}
    B, T = case["B"], case["T"]
    back = case["op"] == "scan_bwd"
    by_group = lambda t: t.view(B, G, D // G, -1)  # noqa: E731
    h = d64("h0").clone() if s["h0"] is not None else torch.zeros(B, D, N, device="cuda",
                                                                  dtype=torch.float64)
    kept = torch.empty(T + 1, B, D, N, device="cuda", dtype=torch.float64) if back else None
    y = torch.empty(B, T, D, device="cuda", dtype=torch.float64)
    clears = s["starts"].any(0).tolist() if s["starts"] is not None else [False] * T
    for t in range(T):
        if clears[t]:
            h = h.clone()
            h[s["starts"][:, t]] = 0.0
        if back:
            kept[t] = h                                   # after a document's clearing
        ut, xt = u[:, t], s["x"][:, t].double()
        h = torch.exp(ut[..., None] * A) * h
        by_group(h).add_(by_group(ut * xt) * s["B"][:, t, :, None].double())
        y[:, t] = (by_group(h) @ s["C"][:, t, :, :, None].double()).view(B, D)
    x = d64("x")
    gated = y + skip * x
    if not back:
        return {"y": gated if s["z"] is None else gated * _act64(d64("z")), "h": h}
    kept[T] = h
    p = d64("dy") if s["z"] is None else d64("dy") * _act64(d64("z"))
    out = {n: torch.zeros(s[n].shape, device="cuda", dtype=torch.float64)
           for n in ("x", "dt", "A", "B", "C")}
    E = d64("dhT").clone() if s["dhT"] is not None else torch.zeros_like(h)
    du = torch.empty_like(u)
    for t in range(T - 1, -1, -1):
        ut, xt, pt = u[:, t], x[:, t], p[:, t]
        bt, ct = s["B"][:, t, :, None].double(), s["C"][:, t, :, None].double()
        a = torch.exp(ut[..., None] * A)
        ah = a * kept[t]
        by_group(E).add_(by_group(pt) * ct)
        q = (by_group(E) * bt).sum(-1).view(B, D)
        now = ah + (by_group(ut * xt) * bt).view(B, D, N)
        out["C"][:, t] = (by_group(now) * by_group(pt)).sum(2)
        out["B"][:, t] = (by_group(E) * by_group(ut * xt)).sum(2)
        w = E * ah
        out["A"] += (w * ut[..., None]).sum(0)
        du[:, t] = (w * A).sum(-1) + xt * q
        out["x"][:, t] = ut * q + skip * pt
        E = a * E
        if clears[t]:
            E[s["starts"][:, t]] = 0.0
    out["dt"] = du / (1.0 + torch.exp(-raw))
    out["dt_bias"] = out["dt"].sum((0, 1))
    out["skip"] = (p * x).sum((0, 1))
    out["h0"] = E
    if s["z"] is not None:
        out["z"] = d64("dy") * gated * _act64_slope(d64("z"))
    return out


def _exact_norms(case, s):
    D = case["D"]
    x, post, pre = s["x"].double(), s["post"].double(), s["pre"].double()
    scale = s["scale"].double() if s["scale"] is not None else torch.ones(D, device="cuda",
                                                                          dtype=torch.float64)
    gate = 1.0 / (1.0 + torch.exp(-s["gate"].double())) if s["gate"] is not None else 1.0
    rms_x = torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS)
    unit = x / rms_x
    if case["op"] == "norms_fwd":
        exact = s["residual"].double() + scale * gate * unit * post
        r = exact.to(s["x"].dtype).double()     # stored in the inputs' type, and normed from there
        return {"y": r / torch.sqrt((r ** 2).mean(-1, keepdim=True) + EPS) * pre,
                "residual": exact}
    r, dy = s["sum"].double(), s["dy"].double()
    rms_r = torch.sqrt((r ** 2).mean(-1, keepdim=True) + EPS)
    n = r / rms_r
    dn = dy * pre
    dr = s["dres"].double() + (dn - n * (dn * n).mean(-1, keepdim=True)) / rms_r
    du = dr * scale * gate
    dun = du * post
    out = {"pre": torch.einsum("rd,rd->d", dy, n), "residual": dr, "post": (du * unit).sum(0)}
    if s["scale"] is not None:
        out["scale"] = (dr * gate * unit * post).sum(0)
    if s["gate"] is not None:
        out["gate"] = dr * scale * unit * post * gate * (1.0 - gate)
    out["x"] = (dun - unit * (dun * unit).mean(-1, keepdim=True)) / rms_x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("conv"):
        return _exact_conv(case, s)
    if case["op"].startswith("scan"):
        return _exact_scan(case, s)
    return _exact_norms(case, s)
