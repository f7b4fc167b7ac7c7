"""GPU parity of the block operators through the public entry points against the float64
oracle (oracle/block.py).

Bars, from the arithmetic:
* an element of a result in bf16 is rounded once: 2^-8 of the value; in fp32 2^-22 (the
  last few operations' 2^-24 each).
* before that, convolution: sums of K + 1 products in fp32, and an exponential of 2^-22 in
  the activation: 1e-6 of the largest element.
* state space: a decay is an exponential of 2^-22, and a state that keeps M tokens passes M
  of them, so that it is off by M 2^-22 at most, T tokens' at most; the products' sums add
  2e-6. Of the largest element (of the 2-norm for sums over tokens): 2e-6 + T 2^-22. The
  step sizes are 2^-21 at worst, which is part of it.
* norms: a few 2^-24 and the sigmoid's 2^-22: 2e-6 of the largest element; their sums over
  rows 1e-5 of the 2-norm.
"""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from gated_delta_rule_10_gb300 import block as wrappers
from oracle import block

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, ref, slack, what=""):
    """Element by element: one rounding to got's type, and `slack` of the largest."""
    ref = np.asarray(ref)
    band = (2.0 ** -8 if got.dtype == BF else 2.0 ** -22) * np.abs(ref)
    top = np.abs(ref).max()
    d = np.abs(f64(got) - ref)
    assert (d <= band + slack * top).all(), (what, float((d - band).max() / top), slack)


def off(got, ref):
    n = np.linalg.norm(ref)
    d = np.linalg.norm(f64(got) - ref)
    return d / n if n else d


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def ids(v):
    return "x".join(map(str, v)) if isinstance(v, tuple) else str(v)


# ------------------------------------------------------------------ short convolution

def conv_inputs(B, T, D, K, dtype, seed=0, packed=False, state=True, bias=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = {"x": rnd(gen, B, T, D).to(dtype), "weight": rnd(gen, D, K) * 0.5,
         "bias": rnd(gen, D) if bias else None,
         "state": rnd(gen, B, K - 1, D).to(dtype) if state else None,
         "dy": rnd(gen, B, T, D).to(dtype), "dstate": rnd(gen, B, K - 1, D).to(dtype),
         "starts": None}
    if packed:
        x["starts"] = torch.rand(B, T, generator=gen, device="cuda") < 0.2
        for t in (0, 7, 8, 9, 31, 32, 255, 256):     # the edges of runs
            if t < T:
                x["starts"][-1, t] = True
    return x


def check_conv(x, silu=True):
    B = x["x"].shape[0]
    y, last = gdr.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state"], starts=x["starts"],
                                 silu=silu)
    g = gdr.short_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], x["state"], x["dstate"],
                           starts=x["starts"], silu=silu)
    row = lambda n, b: None if x[n] is None else f64(x[n][b])  # noqa: E731
    w, bias = f64(x["weight"]), f64(x["bias"])
    dw, db = 0, 0
    refs = {n: [] for n in ("y", "last", "x", "state")}
    for b in range(B):
        ry, rl = block.short_conv(row("x", b), w, bias, row("state", b), row("starts", b), silu)
        r = block.short_conv_gradients(row("dy", b), row("x", b), w, bias, row("state", b),
                                       row("dstate", b), row("starts", b), silu)
        dw, db = dw + r["weight"], db + r["bias"]
        for n, v in (("y", ry), ("last", rl), ("x", r["x"]), ("state", r["state"])):
            refs[n].append(v)
    near(y, np.stack(refs["y"]), 1e-6, "y")
    assert np.array_equal(f64(last), np.stack(refs["last"]))
    near(g["x"], np.stack(refs["x"]), 2e-6, "dx")
    near(g["state"], np.stack(refs["state"]), 2e-6, "dstate")
    assert off(g["weight"], dw) <= 1e-5 and off(g["bias"], db) <= 1e-5
    return y, last, g


CONV = [(1, 1, 8, 4), (2, 2, 16, 4), (3, 3, 24, 3), (1, 9, 136, 4), (2, 31, 64, 2), (1, 33, 8, 4),
        (2, 257, 264, 4), (2, 300, 40, 3), (1, 1000, 128, 4)]


@DTYPES
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("shape", CONV, ids=ids)
def test_conv(shape, packed, dtype):
    check_conv(conv_inputs(*shape, dtype, seed=sum(shape), packed=packed))


@DTYPES
def test_conv_without_bias_state_or_activation(dtype):
    check_conv(conv_inputs(2, 50, 32, 4, dtype, 3, packed=True, state=False, bias=False), silu=False)


def test_conv_every_token_starts():
    x = conv_inputs(2, 40, 16, 4, BF, 4)
    x["starts"] = torch.ones(2, 40, dtype=torch.uint8, device="cuda")
    check_conv(x)


def test_conv_long_runs():
    """Enough channels for the longest runs, both ways."""
    B, T, D, K = 2, 1100, 8192, 4
    x = conv_inputs(B, T, D, K, BF, 5, packed=True)
    y, _ = gdr.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state"], starts=x["starts"])
    g = gdr.short_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], x["state"], x["dstate"],
                           starts=x["starts"])
    part = slice(4000, 4064)
    dw = 0
    for b in range(B):
        args = (f64(x["x"][b, :, part]), f64(x["weight"][part]), f64(x["bias"][part]),
                f64(x["state"][b, :, part]))
        r, _ = block.short_conv(*args, f64(x["starts"][b]))
        near(y[b, :, part], r, 1e-6)
        r = block.short_conv_gradients(f64(x["dy"][b, :, part]), *args, f64(x["dstate"][b, :, part]),
                                       f64(x["starts"][b]))
        near(g["x"][b, :, part], r["x"], 2e-6)
        near(g["state"][b, :, part], r["state"], 2e-6)
        dw = dw + r["weight"]
    assert off(g["weight"][part], dw) <= 1e-5


@DTYPES
def test_conv_in_pieces_and_steps(dtype):
    """A prompt in two calls and single tokens is one prompt, bit for bit."""
    x = conv_inputs(3, 60, 72, 4, dtype, 6)
    w, b = x["weight"], x["bias"]
    y, last = gdr.short_conv_fwd(x["x"], w, b, x["state"])
    a, s = gdr.short_conv_fwd(x["x"][:, :25].contiguous(), w, b, x["state"])
    c, s = gdr.short_conv_fwd(x["x"][:, 25:40].contiguous(), w, b, s)
    steps = []
    for t in range(40, 60):
        at = x["x"][:, t]                             # a strided row
        steps.append(gdr.short_conv_step(at, w, b, s))
    got = torch.cat([a, c, torch.stack(steps, 1)], 1)
    near(got, f64(y), 1e-6)
    assert torch.equal(s, last)


def test_conv_takes_a_part_of_a_projection_and_another_stream():
    x = conv_inputs(2, 130, 64, 4, BF, 7, packed=True)
    p = torch.zeros(2, 130, 200, device="cuda", dtype=BF)
    p[..., 72:136] = x["x"]
    part = {**x, "x": p[..., 72:136]}
    y, last, g = check_conv(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, l2 = gdr.short_conv_fwd(part["x"], x["weight"], x["bias"], x["state"], starts=x["starts"],
                                stream=side)
    g2 = gdr.short_conv_bwd(x["dy"], part["x"], x["weight"], x["bias"], x["state"], x["dstate"],
                            starts=x["starts"], stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(last, l2)
    assert all(torch.equal(g[n], g2[n]) for n in g)


def test_conv_values_of_another_document_do_not_matter():
    """NaN and infinity behind a start, in the state too, reach nothing."""
    x = conv_inputs(1, 20, 16, 4, BF, 8)
    x["starts"] = torch.zeros(1, 20, dtype=torch.bool, device="cuda")
    x["starts"][0, 0] = x["starts"][0, 10] = True
    y, last = gdr.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state"], starts=x["starts"])
    x["x"][0, 9] = torch.nan
    x["x"][0, 8] = torch.inf
    x["state"][:] = torch.nan
    y2, l2 = gdr.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state"], starts=x["starts"])
    assert torch.equal(y[:, :8], y2[:, :8]) and torch.equal(y[:, 10:], y2[:, 10:])
    assert torch.equal(last, l2) and torch.isnan(y2[:, 9]).all()
    g = gdr.short_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], x["state"], starts=x["starts"])
    assert torch.isfinite(g["x"][:, 10:]).all() and torch.isfinite(g["x"][:, :5]).all()
    assert torch.all(g["state"] == 0)


def test_conv_gradient_against_differences():
    """fp32: the slope along a random direction."""
    x = conv_inputs(2, 23, 16, 4, F32, 9, packed=True)
    names = ("x", "weight", "bias", "state")

    def loss(v):
        y, s = gdr.short_conv_fwd(v["x"], v["weight"], v["bias"], v["state"], starts=x["starts"])
        return float((y.double() * x["dy"].double()).sum() +
                     (s.double() * x["dstate"].double()).sum())

    g = gdr.short_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], x["state"], x["dstate"],
                           starts=x["starts"])
    e = 1e-2
    for n in names:
        d = torch.randn_like(x[n])
        num = (loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e)
        assert abs(num - float((g[n].double() * d.double()).sum())) <= 1e-2 * float(g[n].norm()), n


# ------------------------------------------------------------------ state space recurrence

def space_inputs(B, T, D, G, N, dtype, seed=0, packed=False, z=True, state=True, skip=True,
                 bias=True, softplus=True, fast=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = {"x": rnd(gen, B, T, D).to(dtype), "B": rnd(gen, B, T, G, N).to(dtype),
         "C": rnd(gen, B, T, G, N).to(dtype), "z": rnd(gen, B, T, D).to(dtype) if z else None,
         "A": -torch.exp(rnd(gen, D, N)) * (8 if fast else 1),
         "skip": rnd(gen, D) if skip else None,
         "h0": rnd(gen, B, D, N) if state else None, "dhT": rnd(gen, B, D, N) if state else None,
         "dy": rnd(gen, B, T, D).to(dtype), "starts": None, "softplus": softplus}
    if softplus:
        x["dt"] = rnd(gen, B, T, D).to(dtype)
        x["dt_bias"] = rnd(gen, D) - 3.0 if bias else None
    else:
        x["dt"] = (0.2 * torch.rand(B, T, D, generator=gen, device="cuda")).to(dtype)
        x["dt_bias"] = 0.1 * torch.rand(D, generator=gen, device="cuda") if bias else None
    if packed:
        x["starts"] = torch.rand(B, T, generator=gen, device="cuda") < 0.02
        for t in (0, 15, 16, 17, 31, 32, 47, 160, 161):      # the edges of tiles
            if t < T:
                x["starts"][-1, t] = True
    return x


KW = ("skip", "z", "dt_bias", "softplus", "starts")


def space_fwd(x, **kw):
    return gdr.state_space_fwd(x["x"], x["dt"], x["A"], x["B"], x["C"], x["h0"],
                               **{n: x[n] for n in KW}, **kw)


def space_bwd(x, **kw):
    return gdr.state_space_bwd(x["dy"], x["x"], x["dt"], x["A"], x["B"], x["C"], x["h0"], x["dhT"],
                               **{n: x[n] for n in KW}, **kw)


def space_oracle(x, b, backward):
    row = lambda n: None if x[n] is None else f64(x[n][b])  # noqa: E731
    args = (row("x"), row("dt"), f64(x["A"]), row("B"), row("C"), row("h0"))
    rest = (f64(x["skip"]), row("z"), f64(x["dt_bias"]), x["softplus"], row("starts"))
    if backward:
        return block.state_space_gradients(row("dy"), *args, row("dhT"), *rest)
    y, h = block.state_space(*args, *rest)
    return y, h[-1]


def check_space(x, rows=None):
    B, T = x["x"].shape[:2]
    tol = 2e-6 + T * 2.0 ** -22
    y, hT = space_fwd(x)
    g = space_bwd(x)
    sums = {n: 0 for n in ("A", "skip", "dt_bias")}
    for b in range(B):
        ry, rh = space_oracle(x, b, False)
        near(y[b], ry, tol, "y")
        near(hT[b], rh, tol, "hT")
        r = space_oracle(x, b, True)
        for n in sums:
            sums[n] = sums[n] + r[n]
        for n in ("x", "dt", "B", "C", "h0") + (("z",) if x["z"] is not None else ()):
            assert g[n].dtype == (F32 if n == "h0" else x["x"].dtype)
            near(g[n][b], r[n], tol, "d" + n)
    for n, ref in sums.items():
        if n != "A" and x[n] is None:
            assert g[n] is None
        else:
            assert off(g[n], ref) <= tol + 1e-5, n
    return y, hT, g


# one token, tiles of 16 and 32 and their edges, channels that fill a CTA and do not,
# groups, every number of states; lengths that are cut into segments
SPACE = [(1, 1, 8, 1, 16), (2, 15, 24, 1, 16), (1, 16, 64, 2, 8), (2, 17, 136, 1, 16), (1, 33, 16, 2, 64),
         (2, 70, 48, 3, 32), (1, 130, 264, 1, 8), (1, 200, 40, 1, 64), (2, 300, 96, 3, 16),
         (1, 517, 72, 1, 32)]


@DTYPES
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("shape", SPACE, ids=ids)
def test_space(shape, packed, dtype):
    check_space(space_inputs(*shape, dtype, seed=sum(shape), packed=packed))


@DTYPES
@pytest.mark.parametrize("off_", ["z", "skip", "state", "bias", "softplus", "all"])
def test_space_without(off_, dtype):
    kw = {n: False for n in ("z", "skip", "state", "bias", "softplus") if off_ in (n, "all")}
    check_space(space_inputs(2, 90, 40, 1, 16, dtype, 5, packed=True, **kw))


@DTYPES
def test_space_fast_decays(dtype):
    """Decays down to zero within a token."""
    x = space_inputs(1, 150, 32, 1, 16, dtype, 6, fast=True)
    x["dt"] = x["dt"] * 8
    check_space(x)


@DTYPES
@pytest.mark.parametrize("T", [40, 700])
def test_space_extreme_step_sizes(T, dtype):
    """Steps of zero (dt of minus infinity, of the type's lowest value: tokens that leave the
    state as it is) and steps after which nothing of the state is left."""
    x = space_inputs(2, T, 24, 1, 16, dtype, 12)
    x["dt"][0, 3::7] = -torch.inf
    x["dt"][0, 5::11] = torch.finfo(dtype).min
    x["dt"][1, ::2] = -200.0
    x["dt"][1, 1::8] = 1e3
    x["x"][1, 1::8] = 1e-3
    check_space(x)


def test_space_every_token_starts():
    x = space_inputs(1, 70, 16, 1, 16, BF, 7)
    x["starts"] = torch.ones(1, 70, dtype=torch.uint8, device="cuda")
    _, _, g = check_space(x)
    assert torch.all(g["h0"] == 0) and torch.all(g["A"] == 0)


@DTYPES
@pytest.mark.parametrize("N,G", [(16, 1), (8, 2), (64, 1)])
def test_space_segments(N, G, dtype):
    """Long sequences of few channels: many segments, from a state, with starts in some."""
    x = space_inputs(1, 2100, 16 * G, G, N, dtype, 8)
    x["starts"] = torch.zeros(1, 2100, dtype=torch.bool, device="cuda")
    x["starts"][0, 700] = x["starts"][0, 1500] = True
    check_space(x)


def test_space_runs_are_identical_and_one_buffer_for_states():
    x = space_inputs(1, 900, 128, 1, 16, BF, 9, packed=True)
    y, hT = space_fwd(x)
    g = space_bwd(x)
    for _ in range(3):
        h = x["h0"].clone()
        y2, h2 = gdr.state_space_fwd(x["x"], x["dt"], x["A"], x["B"], x["C"], h, hT=h,
                                     **{n: x[n] for n in KW})
        assert h2 is h and torch.equal(y, y2) and torch.equal(hT, h)
        g2 = space_bwd(x)
        assert all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("T", [40, 900])
def test_space_state_gradients_in_one_buffer(T):
    """dhT and dh0 may be one buffer, whole and cut into segments."""
    x = space_inputs(1, T, 64, 1, 16, BF, 10)
    g = space_bwd(x)
    s = wrappers._space_shape(x["x"], x["dt"], x["A"], x["B"], x["C"], x["skip"], x["z"],
                              x["dt_bias"], True, 2)
    ws = torch.empty(gdr.state_space_bwd_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    both = x["dhT"].clone()
    out = {n: torch.empty_like(v) for n, v in g.items()}
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = wrappers._lib().gdr_state_space_bwd(
        ctypes.byref(s), *(p(x[n]) for n in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias",
                                             "starts", "h0", "dy")), p(both),
        *(p(out[n]) for n in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias")), p(both), p(ws),
        ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(both, g["h0"]) and torch.equal(out["x"], g["x"])


@DTYPES
def test_space_takes_parts_of_projections_and_another_stream(dtype):
    x = space_inputs(2, 150, 64, 2, 16, dtype, 11, packed=True)
    p = torch.zeros(2, 150, 328, device="cuda", dtype=dtype)
    far = dict(x)
    at = 8
    for n in ("x", "dt", "z"):
        far[n] = p[..., at:at + 64]
        at += 64
    for n in ("B", "C"):
        far[n] = p[..., at:at + 32].unflatten(-1, (2, 16))
        at += 32
    for n in ("x", "dt", "z", "B", "C"):
        far[n].copy_(x[n])
    y, hT = space_fwd(x)
    g = space_bwd(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, h2 = space_fwd(far, stream=side)
    g2 = space_bwd(far, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(hT, h2)
    assert all(torch.equal(g[n], g2[n]) for n in g)


def test_space_offsets_past_32_bits():
    """Tokens 60 million elements apart: the last ones lie past 2^31."""
    T, step = 40, 60_000_000
    base = torch.empty(T * step, dtype=BF, device="cuda")
    x = space_inputs(1, T, 64, 1, 16, BF, 12)
    far = dict(x)
    for i, n in enumerate(("x", "dt", "z")):
        far[n] = base.as_strided((1, T, 64), (T * step, step, 1), 64 * i)
    for i, n in enumerate(("B", "C")):
        far[n] = base.as_strided((1, T, 1, 16), (T * step, step, 16, 1), 192 + 16 * i)
    for n in ("x", "dt", "z", "B", "C"):
        far[n].copy_(x[n])
    assert all(torch.equal(a, b) for a, b in zip(space_fwd(far), space_fwd(x)))
    a, b = space_bwd(far), space_bwd(x)
    assert all(torch.equal(a[n], b[n]) for n in a)
    w, bias = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda")
    for f in (lambda v: gdr.short_conv_fwd(v, w, bias)[0],
              lambda v: gdr.short_conv_bwd(x["dy"], v, w, bias)["x"]):
        assert torch.equal(f(far["x"]), f(x["x"]))


def test_space_values_of_another_document_do_not_matter():
    x = space_inputs(1, 120, 32, 1, 16, BF, 13)
    x["starts"] = torch.zeros(1, 120, dtype=torch.bool, device="cuda")
    x["starts"][0, 50] = True
    y, hT = space_fwd(x)
    g = space_bwd(x)
    x["x"][0, 30, 5] = torch.nan
    x["x"][0, 31, 7] = torch.inf
    y2, h2 = space_fwd(x)
    g2 = space_bwd(x)
    assert torch.equal(y[:, 50:], y2[:, 50:]) and torch.equal(hT, h2)
    assert torch.equal(y[:, :30], y2[:, :30]) and torch.isnan(y2[0, 30:50, 5]).all()
    for n in ("x", "dt", "z", "B", "C"):
        assert torch.equal(g[n][:, 50:], g2[n][:, 50:]), n
    # the gradients of channels that did not meet it
    assert torch.equal(g["x"][..., 8:], g2["x"][..., 8:])


@DTYPES
@pytest.mark.parametrize("N,D,G,S", [(1, 8, 1, 16), (3, 136, 1, 8), (5, 48, 2, 64), (40, 264, 3, 32),
                                     (7, 1024, 1, 16)])
def test_space_step(N, D, G, S, dtype):
    x = space_inputs(N, 1, D, G, S, dtype, N + D)
    state = x["h0"].clone()
    y = gdr.state_space_step(x["x"][:, 0], x["dt"][:, 0], x["A"], x["B"][:, 0], x["C"][:, 0], state,
                             skip=x["skip"], z=x["z"][:, 0], dt_bias=x["dt_bias"])
    for b in range(N):
        ry, rh = space_oracle(x, b, False)
        near(y[b], ry[0], 2e-6)
        near(state[b], rh, 2e-6)


def test_space_step_sequences_apart():
    """Parts of projections, more sequences than a warp has channels, widths that end inside
    a warp."""
    N, D, S = 37, 200, 16
    x = space_inputs(N, 1, D, 1, S, BF, 21)
    p = torch.zeros(N, 8 + 3 * D + 2 * S, device="cuda", dtype=BF)
    part = lambda at, n, like: p[:, at:at + n].copy_(like)  # noqa: E731
    parts = [part(8 + i * D, D, x[n][:, 0]) for i, n in enumerate(("x", "dt", "z"))]
    bc = [part(8 + 3 * D + i * S, S, x[n][:, 0, 0]).unsqueeze(1) for i, n in enumerate(("B", "C"))]
    s1, s2 = x["h0"].clone(), x["h0"].clone()
    kw = dict(skip=x["skip"], dt_bias=x["dt_bias"])
    y1 = gdr.state_space_step(parts[0], parts[1], x["A"], bc[0], bc[1], s1, z=parts[2], **kw)
    y2 = gdr.state_space_step(x["x"][:, 0], x["dt"][:, 0], x["A"], x["B"][:, 0], x["C"][:, 0], s2,
                              z=x["z"][:, 0], **kw)
    assert torch.equal(y1, y2) and torch.equal(s1, s2)
    for b in (0, 17, N - 1):
        ry, rh = space_oracle(x, b, False)
        near(y1[b], ry[0], 2e-6)
        near(s1[b], rh, 2e-6)


@pytest.mark.parametrize("shape", [(3, 40, 4096, 1, 16), (4, 300, 2048, 1, 16), (2, 64, 1024, 2, 64)],
                         ids=ids)
def test_space_wide_layers(shape):
    """Channels of many CTAs, uncut and cut: a few of them, and all sums over channels, from
    the oracle on those channels alone and from the others' own calls."""
    B, T, D, G, N = shape
    x = space_inputs(*shape, BF, 22, packed=True)
    y, hT = space_fwd(x)
    g = space_bwd(x)
    each = D // G
    tol = 2e-6 + T * 2.0 ** -22
    cut = slice(each - 8, each)                      # the last channels of the first group
    sub = {n: (v if v is None or not torch.is_tensor(v) else
               v[..., cut].contiguous() if n in ("x", "dt", "z", "dy") else
               v[cut].contiguous() if n in ("A", "skip", "dt_bias") else
               v[:, cut].contiguous() if n in ("h0", "dhT") else
               v[:, :, :1].contiguous() if n in ("B", "C") else v) for n, v in x.items()}
    for b in range(B):
        ry, rh = space_oracle(sub, b, False)
        near(y[b, :, cut], ry, tol)
        near(hT[b, cut], rh, tol)
        r = space_oracle(sub, b, True)
        for n in ("x", "dt", "z"):
            near(g[n][b, :, cut], r[n], tol, n)
        near(g["h0"][b, cut], r["h0"], tol)
    # dB and dC are sums over channels: of the parts' own calls, in fp32
    total = {n: torch.zeros(B, T, 1, N, device="cuda", dtype=torch.float64) for n in ("B", "C")}
    for at in range(0, each, 512):
        part = slice(at, min(at + 512, each))
        sub = {n: (v if v is None or not torch.is_tensor(v) else
                   v[..., part].float().contiguous() if n in ("x", "dt", "z", "dy") else
                   v[part].contiguous() if n in ("A", "skip", "dt_bias") else
                   v[:, part].contiguous() if n in ("h0", "dhT") else
                   v[:, :, :1].float().contiguous() if n in ("B", "C") else v) for n, v in x.items()}
        p = space_bwd(sub)
        for n in total:
            total[n] += p[n].double()
    for n in total:
        near(g[n][:, :, :1], f64(total[n]), 2 * tol, "d" + n)


def test_space_prompt_then_steps_is_one_prompt():
    x = space_inputs(2, 80, 48, 1, 16, F32, 14)
    y, hT = space_fwd(x)
    cut = {n: (v[:, :60].contiguous() if torch.is_tensor(v) and v.dim() > 2 and v.shape[1] == 80
               else v) for n, v in x.items()}
    a, h = space_fwd(cut)
    out = [a]
    for t in range(60, 80):
        out.append(gdr.state_space_step(x["x"][:, t], x["dt"][:, t], x["A"], x["B"][:, t],
                                        x["C"][:, t], h, skip=x["skip"], z=x["z"][:, t],
                                        dt_bias=x["dt_bias"])[:, None])
    near(torch.cat(out, 1), f64(y), 2e-6 + 80 * 2.0 ** -22)
    near(h, f64(hT), 2e-6 + 80 * 2.0 ** -22)


def test_space_gradient_against_differences():
    x = space_inputs(1, 37, 16, 1, 8, F32, 15, packed=True)

    def loss(v):
        y, h = space_fwd(v)
        return float((y.double() * x["dy"].double()).sum() + (h.double() * x["dhT"].double()).sum())

    g = space_bwd(x)
    e = 2e-3
    for n in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0"):
        d = torch.randn_like(x[n])
        num = (loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e)
        assert abs(num - float((g[n].double() * d.double()).sum())) <= 1e-2 * float(g[n].norm()), n


# ------------------------------------------------------------------ norms around a block

NORMS = [(1, 8), (3, 64), (5, 256), (2, 264), (9, 520), (4, 1032), (7, 2048), (3, 4104), (2, 8192),
         (700, 136)]


def norms_inputs(rows, D, dtype, seed, gate=True, scale=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = {n: (k * rnd(gen, rows, D)).to(dtype) for n, k in (("x", 3), ("residual", 2), ("gate", 2),
                                                            ("dy", 1), ("dres", 1))}
    x.update(post=1 + 0.2 * rnd(gen, D), pre=1 + 0.2 * rnd(gen, D), scale=0.5 + 0.2 * rnd(gen, D))
    if not gate:
        x["gate"] = None
    if not scale:
        x["scale"] = None
    return x


@DTYPES
@pytest.mark.parametrize("gate,scale", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("rows,D", NORMS)
def test_norms(rows, D, gate, scale, dtype):
    x = norms_inputs(rows, D, dtype, rows + D, gate, scale)
    y, r = gdr.block_norms(x["x"], x["residual"], x["post"], x["pre"], 1e-5, gate=x["gate"],
                           scale=x["scale"])
    near(r, block.block_sum(*(f64(x[n]) for n in ("x", "residual", "post", "gate", "scale")), 1e-5),
         2e-6)
    near(y, block.pre_norm(f64(r), f64(x["pre"]), 1e-5), 2e-6)
    run = lambda **kw: gdr.block_norms_bwd(x["dy"], x["x"], r, x["post"], x["pre"], 1e-5,  # noqa: E731
                                           gate=x["gate"], scale=x["scale"], **kw)
    for dres in (x["dres"], None):
        g = run(dres=dres)
        ref = block.block_norms_gradients(f64(x["dy"]), f64(x["x"]), f64(r), f64(x["post"]),
                                          f64(x["pre"]), f64(x["gate"]), f64(x["scale"]), f64(dres),
                                          1e-5)
        for n in ("x", "residual", "gate"):
            if n == "gate" and not gate:
                assert g[n] is None
            else:
                near(g[n], ref[n], 4e-6, n)
        for n in ("post", "pre", "scale"):
            if n == "scale" and not scale:
                assert g[n] is None
            else:
                assert off(g[n], ref[n]) <= 1e-5, n
    again = run(dres=None)
    assert all(g[n] is None or torch.equal(g[n], again[n]) for n in g)


def test_norms_in_place_empty_and_non_finite():
    x = norms_inputs(9, 256, BF, 4)
    call = lambda v, **kw: gdr.block_norms(v["x"], v["residual"], x["post"], x["pre"],  # noqa: E731
                                           gate=v["gate"], scale=x["scale"], **kw)
    y, r = call(x)
    for out, res in (("x", "residual"), ("gate", "x"), ("residual", "gate")):
        v = {n: x[n].clone() for n in ("x", "residual", "gate")}
        y2, r2 = call(v, out=v[out], residual_out=v[res])
        assert y2 is v[out] and torch.equal(y, y2) and torch.equal(r, r2)
    e = {n: x[n][:0] for n in ("x", "residual", "gate")}
    assert call(e)[0].shape == (0, 256)
    g = gdr.block_norms_bwd(e["x"], e["x"], e["x"], x["post"], x["pre"], gate=e["gate"],
                            scale=x["scale"])
    assert all(torch.all(g[n] == 0) for n in ("post", "pre", "scale"))
    bad = {n: x[n].clone() for n in ("x", "residual", "gate")}
    bad["x"][2, 200] = torch.nan
    bad["gate"][5, 3] = torch.nan
    y2, r2 = call(bad)
    assert torch.isnan(y2[2]).all() and torch.isnan(r2[2]).all()
    assert torch.isnan(y2[5]).all() and torch.isnan(r2[5, 3]) and torch.equal(r2[5, 4:], r[5, 4:])
    keep = [0, 1, 3, 4, 6, 7, 8]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(r[keep], r2[keep])


def test_norms_gradient_against_differences():
    x = norms_inputs(6, 64, F32, 3)

    def loss(v):
        y, r = gdr.block_norms(v["x"], v["residual"], v["post"], v["pre"], gate=v["gate"],
                               scale=v["scale"])
        return float((y.double() * x["dy"].double()).sum() + (r.double() * x["dres"].double()).sum())

    _, r = gdr.block_norms(x["x"], x["residual"], x["post"], x["pre"], gate=x["gate"],
                           scale=x["scale"])
    g = gdr.block_norms_bwd(x["dy"], x["x"], r, x["post"], x["pre"], gate=x["gate"],
                            scale=x["scale"], dres=x["dres"])
    e = 1e-2
    for n in ("x", "residual", "gate", "post", "pre", "scale"):
        d = torch.randn_like(x[n])
        num = (loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e)
        assert abs(num - float((g[n].double() * d.double()).sum())) <= 1e-2 * float(g[n].norm()), n


# ------------------------------------------------------------------ together

def test_a_block_captured_and_replayed():
    """Norms, convolution, recurrence and norms as a block runs them, captured into a graph and
    replayed on new inputs: the same bits as the calls by themselves."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    B, T, D, N = 2, 600, 256, 16
    x, res = rnd(gen, B, T, D).to(BF), rnd(gen, B, T, D).to(BF)
    w, one = rnd(gen, D, 4), torch.ones(D, device="cuda")
    A, bias = -torch.exp(rnd(gen, D, N)), rnd(gen, D) - 3.0
    dt = rnd(gen, B, T, D).to(BF)
    bc = rnd(gen, B, T, 2, N).to(BF)
    dy = rnd(gen, B, T, D).to(BF)

    def run():
        y, r = gdr.block_norms(x, res, one, one, gate=dy)
        c, cs = gdr.short_conv_fwd(y, w)
        space = (c, dt, A, bc[:, :, :1], bc[:, :, 1:])
        o, h = gdr.state_space_fwd(*space, skip=one, z=y, dt_bias=bias)
        out, r2 = gdr.block_norms(o, r, one, one)
        back = gdr.block_norms_bwd(dy, o, r2, one, one)
        g = gdr.state_space_bwd(back["x"], *space, skip=one, z=y, dt_bias=bias)
        gc = gdr.short_conv_bwd(g["x"], y, w)
        gn = gdr.block_norms_bwd(gc["x"], x, r, one, one, gate=dy, dres=back["residual"])
        return [out, r2, h, cs] + [v for d in (back, g, gc, gn) for v in d.values() if v is not None]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in (1, 2):
        x.copy_(rnd(torch.Generator(device="cuda").manual_seed(seed), B, T, D))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, run()))
