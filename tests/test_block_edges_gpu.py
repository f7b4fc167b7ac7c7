"""GPU tests of the block operators at the edges of what their header allows, against the float64
oracle. Bars as in test_block_gpu.py, or derived at the test."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from gated_delta_rule_10_gb300 import block as wrappers
from oracle import block
from test_block_gpu import (BF, DTYPES, F32, check_conv, check_space, conv_inputs, f64, near,
                            norms_inputs, off, rnd, space_bwd, space_fwd, space_inputs, space_oracle)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ short convolution

@DTYPES
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("N,D", [(3, 72), (153, 4096)])       # one and two sequences a thread
def test_conv_steps_move_the_state_in_place(N, D, K, dtype):
    """The state is read and moved on by one kernel: token after token, its rows are the last
    tokens', bit for bit, also of the odd sequence."""
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    w, b = rnd(gen, D, K) * 0.5, rnd(gen, D)
    state = rnd(gen, N, K - 1, D).to(dtype)
    rows = [state[:, k].clone() for k in range(K - 1)]
    for _ in range(6):
        x = rnd(gen, N, D).to(dtype)
        y = gdr.short_conv_step(x, w, b, state)
        rows.append(x)
        s = f64(b) + sum(f64(w[:, k]) * f64(rows[len(rows) - K + k]) for k in range(K))
        near(y, block.silu(s), 1e-6)
        assert all(torch.equal(state[:, k], rows[len(rows) - K + 1 + k]) for k in range(K - 1))


@DTYPES
def test_conv_starts_of_any_address_and_value(dtype):
    """Marks are bytes that are not zero, at any address."""
    x = conv_inputs(1, 300, 64, 4, dtype, 41, packed=True)
    marks = torch.zeros(303, dtype=torch.uint8, device="cuda")
    for by in (1, 2, 3):
        at = marks[by:by + 300].view(1, 300)
        at.copy_(x["starts"].to(torch.uint8) * 0x80)
        check_conv({**x, "starts": at})


@DTYPES
def test_conv_gradients_of_another_document_do_not_matter(dtype):
    """What is not finite behind a start reaches no gradient ahead of it."""
    x = conv_inputs(2, 300, 64, 4, dtype, 48)
    x["starts"] = torch.zeros(2, 300, dtype=torch.bool, device="cuda")
    x["starts"][:, 100] = x["starts"][0, 101] = True
    run = lambda: gdr.short_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], x["state"],  # noqa: E731
                                     x["dstate"], starts=x["starts"])
    g = run()
    x["dy"][:, 102], x["x"][:, 103], x["dstate"][:] = torch.inf, torch.nan, torch.nan
    g2 = run()
    assert torch.equal(g["x"][:, :100], g2["x"][:, :100]) and torch.equal(g["state"], g2["state"])
    assert torch.equal(g["x"][0, :101], g2["x"][0, :101])
    assert torch.isnan(g2["x"][:, 103]).all() and torch.isnan(g2["x"][:, 297:]).all()


def test_conv_offsets_past_32_bits():
    """More than 2^31 elements in and out: the last tokens are those of a call on them alone."""
    T, D, K, tail = 530_000, 4096, 4, 700
    gen = torch.Generator(device="cuda").manual_seed(42)
    x, dy = (torch.randn(1, T, D, generator=gen, device="cuda", dtype=BF) for _ in range(2))
    w, b = rnd(gen, D, K) * 0.5, rnd(gen, D)
    y, last = gdr.short_conv_fwd(x, w, b)
    before = x[:, T - tail - K + 1:T - tail].contiguous()
    y2, last2 = gdr.short_conv_fwd(x[:, T - tail:], w, b, before)
    assert torch.equal(y[:, T - tail:], y2) and torch.equal(last, last2)
    dx = gdr.short_conv_bwd(dy, x, w, b)["x"]
    dx2 = gdr.short_conv_bwd(dy[:, T - tail:].contiguous(), x[:, T - tail:], w, b, before)["x"]
    assert torch.equal(dx[:, T - tail:], dx2)


# ------------------------------------------------------------------ state space recurrence

def test_space_long_memories():
    """States that keep thousands of tokens, walked in long pieces. A token's decay is an
    exponential whose error spreads by 0.5 of 2^-24 and is off by at most 0.05 of it on average
    below 2^-8, and the state's rounding spreads by 0.3: 4096 tokens come to sqrt(4096) 0.6 2^-24
    + 4096 0.05 2^-24, 1.5e-5 at worst for a state that keeps them all, and half of it on average
    over states that keep from a part of them to all. With a bias of 0.1, 2.8e-5."""
    B, T, D, N = 8, 4096, 8192, 16
    gen = torch.Generator(device="cuda").manual_seed(31)
    A = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * rnd(gen, D, N))
    dt = (1e-5 * 100.0 ** torch.rand(B, T, D, generator=gen, device="cuda")).to(BF)
    x, h0 = rnd(gen, B, T, D).to(BF), rnd(gen, B, D, N)
    b, c = rnd(gen, B, T, 1, N).to(BF), rnd(gen, B, T, 1, N).to(BF)
    _, hT = gdr.state_space_fwd(x, dt, A, b, c, h0, softplus=False)
    part = slice(4096, 4160)
    h, rate = h0[:, part].double(), A[part].double()
    for t in range(T):
        u = dt[:, t, part].double()
        h = torch.exp(u[..., None] * rate) * h + (u * x[:, t, part].double())[..., None] * \
            b[:, t].double()
    assert float((hT[:, part].double() - h).norm() / h.norm()) <= 7.5e-6


@DTYPES
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("B,T,D", [(1, 40, 64), (1, 900, 64), (64, 20, 4096)])
def test_space_steps_of_zero_keep_the_state(B, T, D, N, dtype):
    """A decay of exactly one: the state and its gradient pass bit for bit, cut or not."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    x, dy = rnd(gen, B, T, D).to(dtype), torch.zeros(B, T, D, dtype=dtype, device="cuda")
    u = torch.zeros_like(x)
    A, b, h0, dhT = (rnd(gen, D, N), rnd(gen, B, T, 1, N).to(dtype), rnd(gen, B, D, N),
                     rnd(gen, B, D, N))
    _, hT = gdr.state_space_fwd(x, u, A, b, b, h0, softplus=False)
    assert torch.equal(hT, h0)
    assert torch.equal(gdr.state_space_bwd(dy, x, u, A, b, b, h0, dhT, softplus=False)["h0"], dhT)
    state = h0.clone()
    gdr.state_space_step(x[:, 0], u[:, 0], A, b[:, 0], b[:, 0], state, softplus=False)
    assert torch.equal(state, h0)


@pytest.mark.parametrize("N,G", [(16, 1), (8, 2), (32, 1), (64, 1)])
@pytest.mark.parametrize("T,starts", [(517, ()), (2100, ()), (2100, (700, 1500))])
def test_space_segments_in_full_precision(T, starts, N, G):
    """What the header says of fp32 (1e-6 of the 2-norm, 5e-6 at worst), doubled, for sequences
    cut into many segments: a term lost at a segment's edge is more than that."""
    x = space_inputs(1, T, 16 * G, G, N, F32, T + N)
    if starts:
        x["starts"] = torch.zeros(1, T, dtype=torch.bool, device="cuda")
        x["starts"][0, list(starts)] = True
    y, hT = space_fwd(x)
    ry, rh = space_oracle(x, 0, False)
    assert off(y[0], ry) <= 1e-5 and off(hT[0], rh) <= 1e-5
    g, r = space_bwd(x), space_oracle(x, 0, True)
    for n in g:
        assert off(g[n] if n in ("A", "skip", "dt_bias") else g[n][0], r[n]) <= 1e-5, n


@pytest.mark.parametrize("N", [8, 16, 64])
@pytest.mark.parametrize("T,at", [(40, 20), (120, 50), (1200, 640), (1200, 777)])
def test_space_what_is_not_finite_stays_in_its_document(T, at, N):
    """Behind a start it reaches no output or gradient ahead of it, and the other way round; the
    start states' gradient and a cleared state among them."""
    x = space_inputs(2, T, 40, 1, N, BF, T + N)
    x["starts"] = torch.zeros(2, T, dtype=torch.bool, device="cuda")
    x["starts"][:, at] = True
    names = ("x", "dt", "z", "B", "C")
    y, hT = space_fwd(x)
    g = space_bwd(x)
    back = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in x.items()}
    back["dy"][:, at], back["x"][:, at + 3], back["C"][:, T - 1] = torch.inf, torch.nan, torch.nan
    back["dt"][:, at + 5], back["dhT"][:] = torch.nan, torch.inf
    y2, _ = space_fwd(back)
    g2 = space_bwd(back)
    assert torch.equal(y[:, :at], y2[:, :at]) and torch.equal(g["h0"], g2["h0"])
    assert all(torch.equal(g[n][:, :at], g2[n][:, :at]) for n in names)
    ahead = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in x.items()}
    ahead["dy"][:, at - 1], ahead["x"][:, 1], ahead["B"][:, 2] = torch.inf, torch.nan, torch.inf
    ahead["dt"][:, 3], ahead["h0"][:] = torch.nan, torch.inf
    y2, h2 = space_fwd(ahead)
    g2 = space_bwd(ahead)
    assert torch.equal(y[:, at:], y2[:, at:]) and torch.equal(hT, h2)
    assert all(torch.equal(g[n][:, at:], g2[n][:, at:]) for n in names)


@DTYPES
@pytest.mark.parametrize("shape", [(1, 70, 64, 8, 64), (2, 33, 240, 10, 8), (1, 45, 24, 3, 32)],
                         ids=str)
def test_space_groups_of_few_channels(shape, dtype):
    check_space(space_inputs(*shape, dtype, sum(shape), packed=True))


@DTYPES
def test_space_starts_of_any_address_and_value(dtype):
    x = space_inputs(1, 300, 64, 1, 16, dtype, 43, packed=True)
    marks = torch.zeros(303, dtype=torch.uint8, device="cuda")
    for by in (1, 3):
        at = marks[by:by + 300].view(1, 300)
        at.copy_(x["starts"].to(torch.uint8) * 0x80)
        check_space({**x, "starts": at})


@DTYPES
def test_space_prompts_of_one_token(dtype):
    """As many batch rows as are allowed, a token each."""
    B, D, N = 65535, 8, 8
    x = space_inputs(B, 1, D, 1, N, dtype, 44)
    y, hT = space_fwd(x)
    g = space_bwd(x)
    v = {n: f64(t[:, 0] if n not in ("A", "skip", "dt_bias", "h0", "dhT") else t)
         for n, t in x.items() if torch.is_tensor(t)}
    u = block.softplus(v["dt"] + v["dt_bias"])
    a = np.exp(u[..., None] * v["A"])
    h = a * v["h0"] + (u * v["x"])[..., None] * v["B"]
    out = (h * v["C"]).sum(-1) + v["skip"] * v["x"]
    near(y[:, 0], out * block.silu(v["z"]), 2e-6)
    near(hT, h, 2e-6)
    p = v["dy"] * block.silu(v["z"])
    e = v["dhT"] + v["C"] * p[..., None]
    near(g["h0"], a * e, 2e-6)
    near(g["z"][:, 0], v["dy"] * out * block.silu_slope(v["z"]), 2e-6)
    near(g["B"][:, 0, 0], (e * (u * v["x"])[..., None]).sum(1), 2e-6)
    assert off(g["A"], (e * a * v["h0"] * u[..., None]).sum(0)) <= 1e-5
    assert off(g["skip"], (p * v["x"]).sum(0)) <= 1e-5


def test_space_a_long_sequence_of_few_channels():
    """A million tokens are their parts one after the other."""
    T, part = 1_000_003, 50_000
    x = space_inputs(1, T, 8, 1, 8, F32, 45)
    x["starts"] = torch.rand(1, T, device="cuda") < 1e-4
    y, hT = space_fwd(x)
    h, ys = x["h0"], []
    for at in range(0, T, part):
        cut = {n: (t[:, at:at + part].contiguous() if torch.is_tensor(t) and t.dim() > 1 and
                   t.shape[1] == T else t) for n, t in x.items()}
        out, h = space_fwd({**cut, "h0": h})
        ys.append(out)
    assert off(y, f64(torch.cat(ys, 1))) <= 1e-5 and off(hT, f64(h)) <= 1e-5


def test_space_offsets_of_outputs_past_32_bits():
    """More than 2^31 elements of every kind: the last documents' values and gradients are those
    of a call on them alone."""
    T, D, N, tail = 530_000, 4096, 8, 400
    gen = torch.Generator(device="cuda").manual_seed(46)
    wide = lambda *s: torch.randn(1, T, *s, generator=gen, device="cuda", dtype=BF)  # noqa: E731
    x = {n: wide(D) for n in ("x", "dt", "z", "dy")}
    x.update(B=wide(1, N), C=wide(1, N), A=-torch.exp(rnd(gen, D, N)), skip=rnd(gen, D),
             dt_bias=rnd(gen, D) - 3.0, h0=None, dhT=None, softplus=True,
             starts=torch.zeros(1, T, dtype=torch.bool, device="cuda"))
    x["starts"][0, T - tail] = True
    last = {n: (t[:, T - tail:].contiguous() if torch.is_tensor(t) and t.dim() > 1 and
                t.shape[1] == T else t) for n, t in x.items()}
    y, hT = space_fwd(x)
    y2, h2 = space_fwd(last)
    tol = 2e-6 + tail * 2.0 ** -22
    near(y[:, T - tail:], f64(y2), 2.0 ** -8 + tol)      # both are rounded
    assert off(hT, f64(h2)) <= 1e-5
    g, g2 = space_bwd(x), space_bwd(last)
    for n in ("x", "dt", "z", "B", "C"):
        near(g[n][:, T - tail:], f64(g2[n]), 2.0 ** -8 + tol, n)


# ------------------------------------------------------------------ norms around a block

@DTYPES
@pytest.mark.parametrize("rows,D", [(1, 8), (5, 256), (9, 64), (700, 136), (2437, 256), (8, 256),
                                    (5, 264), (3, 8192)])
def test_norms_without_eps(rows, D, dtype):
    """eps = 0 is allowed, and rows that share a CTA with none add nothing to the weights' sums."""
    x = norms_inputs(rows, D, dtype, rows + D)
    y, r = gdr.block_norms(x["x"], x["residual"], x["post"], x["pre"], 0.0, gate=x["gate"],
                           scale=x["scale"])
    near(r, block.block_sum(*(f64(x[n]) for n in ("x", "residual", "post", "gate", "scale")), 0.0),
         2e-6)
    near(y, block.pre_norm(f64(r), f64(x["pre"]), 0.0), 2e-6)
    g = gdr.block_norms_bwd(x["dy"], x["x"], r, x["post"], x["pre"], 0.0, gate=x["gate"],
                            scale=x["scale"], dres=x["dres"])
    ref = block.block_norms_gradients(*(f64(x[n]) for n in ("dy", "x")), f64(r),
                                      *(f64(x[n]) for n in ("post", "pre", "gate", "scale", "dres")),
                                      0.0)
    for n in ("x", "residual", "gate"):
        near(g[n], ref[n], 4e-6, n)
    for n in ("post", "pre", "scale"):
        assert off(g[n], ref[n]) <= 1e-5, n


@DTYPES
@pytest.mark.parametrize("D", [256, 1032])
def test_norms_closed_and_open_gates(D, dtype):
    """Gates of infinities and of the type's lowest and largest value: zero and one."""
    x = norms_inputs(11, D, dtype, 49)
    low = torch.finfo(dtype)
    for i, v in enumerate((-torch.inf, low.min, torch.inf, low.max, -200.0, 200.0)):
        x["gate"][i] = v
    y, r = gdr.block_norms(x["x"], x["residual"], x["post"], x["pre"], gate=x["gate"],
                           scale=x["scale"])
    for i in (0, 1, 4):
        assert torch.equal(r[i], x["residual"][i])
    with np.errstate(over="ignore"):
        near(r, block.block_sum(*(f64(x[n]) for n in ("x", "residual", "post", "gate", "scale"))),
             2e-6)
        ref = block.block_norms_gradients(f64(x["dy"]), f64(x["x"]), f64(r),
                                          *(f64(x[n]) for n in ("post", "pre", "gate", "scale",
                                                                "dres")))
    g = gdr.block_norms_bwd(x["dy"], x["x"], r, x["post"], x["pre"], gate=x["gate"],
                            scale=x["scale"], dres=x["dres"])
    for n in ("x", "residual", "gate"):
        near(g[n], ref[n], 4e-6, n)
    for n in ("post", "pre", "scale"):
        assert off(g[n], ref[n]) <= 1e-5, n


@DTYPES
@pytest.mark.parametrize("D", [256, 2048, 8192])
def test_norms_gradients_in_place(D, dtype):
    """dx, dgate and dresidual may be any of the inputs of their kind."""
    rows = 1003
    x = norms_inputs(rows, D, dtype, D)
    _, r = gdr.block_norms(x["x"], x["residual"], x["post"], x["pre"], gate=x["gate"],
                           scale=x["scale"])
    ins = {"dy": x["dy"], "dres": x["dres"], "x": x["x"], "gate": x["gate"], "sum": r}
    g = gdr.block_norms_bwd(x["dy"], x["x"], r, x["post"], x["pre"], gate=x["gate"],
                            scale=x["scale"], dres=x["dres"])
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    n = ctypes.c_size_t()
    assert wrappers._lib().gdr_block_norms_bwd_workspace(rows, D, ctypes.byref(n)) == 0
    assert n.value <= ws.numel()
    for to in (("x", "gate", "dres"), ("dy", "sum", "x"), ("sum", "dres", "dy"),
               ("gate", "x", "sum"), ("dres", "dy", "gate")):
        v = {k: t.clone() for k, t in ins.items()}
        flat = {k: torch.empty(D, device="cuda") for k in ("post", "scale", "pre")}
        p = lambda *names: [v[k].data_ptr() for k in names]  # noqa: E731
        st = wrappers._lib().gdr_block_norms_bwd(
            rows, D, gdr.GDR_BF16 if dtype == BF else gdr.GDR_F32, *p("dy", "dres", "x", "gate", "sum"),
            *(x[k].data_ptr() for k in ("post", "scale", "pre")), 1e-6, *p(*to),
            *(flat[k].data_ptr() for k in ("post", "scale", "pre")), ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        torch.cuda.synchronize()
        for k, at in zip(("x", "gate", "residual"), to):
            assert torch.equal(v[at], g[k]), (k, at)
        assert all(torch.equal(flat[k], g[k]) for k in flat)


def test_norms_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are those of a call on them alone."""
    rows, D, tail = 270_000, 8192, 37
    gen = torch.Generator(device="cuda").manual_seed(47)
    wide = lambda: torch.randn(rows, D, generator=gen, device="cuda", dtype=BF)  # noqa: E731
    x, res, gate, dy = (wide() for _ in range(4))
    post, pre = 1 + 0.2 * rnd(gen, D), 1 + 0.2 * rnd(gen, D)
    end = slice(rows - tail, rows)
    y, r = gdr.block_norms(x, res, post, pre, gate=gate)
    y2, r2 = gdr.block_norms(x[end], res[end], post, pre, gate=gate[end])
    assert torch.equal(y[end], y2) and torch.equal(r[end], r2)
    g = gdr.block_norms_bwd(dy, x, r, post, pre, gate=gate)
    g2 = gdr.block_norms_bwd(dy[end], x[end], r[end], post, pre, gate=gate[end])
    assert all(torch.equal(g[n][end], g2[n]) for n in ("x", "gate", "residual"))


# ------------------------------------------------------------------ together

def test_two_calls_at_once():
    """Calls on two streams at the same time give what they give by themselves."""
    a, b = (space_inputs(1, 900, 128, 1, 16, BF, seed, packed=True) for seed in (51, 52))
    c, d = (conv_inputs(2, 700, 256, 4, BF, seed, packed=True) for seed in (53, 54))
    n = norms_inputs(700, 256, BF, 55)

    def run(space, conv):
        y, h = space_fwd(space)
        s, last = gdr.short_conv_fwd(conv["x"], conv["weight"], conv["bias"], conv["state"],
                                     starts=conv["starts"])
        g = gdr.short_conv_bwd(conv["dy"], conv["x"], conv["weight"], conv["bias"], conv["state"],
                               conv["dstate"], starts=conv["starts"])
        k = gdr.block_norms_bwd(n["dy"], n["x"], n["residual"], n["post"], n["pre"],
                                gate=n["gate"], scale=n["scale"])
        return [y, h, s, last, *space_bwd(space).values(), *g.values(), *k.values()]

    alone = [run(a, c), run(b, d)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, (s, args) in enumerate(zip(streams, ((a, c), (b, d)))):
            with torch.cuda.stream(s):
                got[i] = run(*args)
    torch.cuda.synchronize()
    for x, y in zip(alone, got):
        assert all(torch.equal(u, v) for u, v in zip(x, y))
