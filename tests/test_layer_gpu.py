"""GPU parity of the layer operators through the public entry points against the
float64 oracle (oracle/layer.py).

Bars, from the arithmetic:
* bf16 results of the linear attention (o, dq, dk, dv), 2-norm relative 4e-3: every
  term passes one operand rounded to bf16 (2^-9) and the result another (2^-9).
* its fp32 states from bf16 inputs, 1e-5: operands kept to 2^-18 in two bf16 terms,
  fp32 accumulation of 128 tokens per chunk (a few 2^-23).
* fp32 inputs, 1e-5: products of operands kept to 2^-21 and accumulated in fp32 over
  up to 128 terms at 2^-23 each.
* the gate's gradient, 2e-5: both states' error, gathered over the blocks it passes.
* streams (step, norm, rotary): the fp32 arithmetic's few 2^-23, then one rounding to
  bf16, element by element 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from gated_delta_rule_10_gb300.retention import RetentionLayer
from oracle import layer

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 4e-3, F32: 1e-5}
STATE_TOL, GATE_TOL = 1e-5, 2e-5


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def off(got, ref):
    got, n = f64(got), np.linalg.norm(ref)
    assert np.isfinite(got).all()
    return np.linalg.norm(got - ref) / n if n else np.abs(got).max()


def attn_inputs(B, T, H, Hk, dk, dv, dtype, seed=0, decay="token", clears=(), h0=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x = {"q": torch.nn.functional.normalize(r(B, T, Hk, dk), dim=-1).to(dtype),
         "k": torch.nn.functional.normalize(r(B, T, Hk, dk), dim=-1).to(dtype),
         "v": r(B, T, H, dv).to(dtype), "h0": r(B, H, dk, dv) if h0 else None,
         "dO": r(B, T, H, dv).to(dtype), "dhT": r(B, H, dk, dv) if h0 else None}
    if decay == "head":
        x["g"] = -torch.exp(r(H) - 3.0)
    elif decay == "none":
        x["g"] = torch.zeros(B, T, H, device="cuda")
    else:
        g = -torch.nn.functional.softplus(r(B, T, H))
        x["g"] = g / 16 if decay == "slow" else g * (8 if decay == "strong" else 1)
        for t in clears:
            if t < T:
                x["g"][:, t] = -torch.inf if t % 2 else -300.0
    x["scale"] = dk ** -0.5
    return x


def expand(g, B, T, H):
    g = f64(g)
    g = np.where(g <= -104.0, -np.inf, g)      # what clears the state, by definition
    return np.broadcast_to(g, (B, T, H)) if g.ndim == 1 else g


def attn_oracle(x):
    B, T, H, dv = x["v"].shape
    o, hT = np.zeros((B, T, H, dv)), np.zeros((B, H, x["q"].shape[-1], dv))
    args = (f64(x["q"]), f64(x["k"]), f64(x["v"]), expand(x["g"], B, T, H))
    for b, h, (y, S) in layer.heads(layer.decay_recurrence, *args, f64(x["h0"]), scale=x["scale"]):
        o[b, :, h], hT[b, h] = y, S[-1]
    return o, hT


def attn_grad_oracle(x):
    B, T, H, dv = x["v"].shape
    Hk, dk = x["q"].shape[2:]
    out = {"q": np.zeros((B, T, Hk, dk)), "k": np.zeros((B, T, Hk, dk)),
           "v": np.zeros((B, T, H, dv)), "g": np.zeros((B, T, H)), "h0": np.zeros((B, H, dk, dv))}
    args = (f64(x["q"]), f64(x["k"]), f64(x["v"]), expand(x["g"], B, T, H))
    for b, h, y in layer.heads(layer.decay_gradients, *args, f64(x["dO"]), f64(x["h0"]),
                               f64(x["dhT"]), scale=x["scale"]):
        out["q"][b, :, h * Hk // H] += y["q"]
        out["k"][b, :, h * Hk // H] += y["k"]
        out["v"][b, :, h], out["g"][b, :, h], out["h0"][b, h] = y["v"], y["g"], y["h0"]
    if x["g"].dim() == 1:
        out["g"] = out["g"].sum((0, 1))
    return out


def run_fwd(x, **kw):
    o, hT = gdr.decay_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], scale=x["scale"], **kw)
    torch.cuda.synchronize()
    return o, hT


def run_bwd(x, **kw):
    out = gdr.decay_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dhT"],
                              scale=x["scale"], **kw)
    torch.cuda.synchronize()
    return out


def check_fwd(x):
    o, hT = run_fwd(x)
    ro, rh = attn_oracle(x)
    assert off(o, ro) <= TOL[x["q"].dtype]
    assert off(hT, rh) <= STATE_TOL


def check_bwd(x):
    got, ref = run_bwd(x), attn_grad_oracle(x)
    for n in ("q", "k", "v"):
        assert got[n].dtype == x["q"].dtype
        assert off(got[n], ref[n]) <= TOL[x["q"].dtype], n
    assert off(got["h0"], ref["h0"]) <= STATE_TOL
    assert off(got["g"], ref["g"]) <= GATE_TOL


# lengths around the chunks (64, 128) and blocks (32), segments (several chunks), one
# token; clears at the edges of blocks and chunks, next to one another, everywhere
CLEARS = (0, 31, 32, 33, 63, 64, 127, 128, 130, 131, 200)
SHAPES = [(1, 1, 1, 1, 64, 64), (2, 2, 2, 1, 128, 64), (1, 31, 3, 3, 64, 128),
          (2, 127, 2, 2, 128, 128), (1, 128, 4, 2, 64, 64), (1, 129, 2, 1, 128, 128),
          (1, 700, 2, 2, 128, 64), (1, 1100, 3, 1, 64, 128)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay,clears", [("token", ()), ("slow", CLEARS), ("head", ())],
                         ids=["token", "clears", "head"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_attention_forward(shape, decay, clears, dtype):
    check_fwd(attn_inputs(*shape, dtype, seed=sum(shape), decay=decay, clears=clears,
                          h0=shape[1] % 2 == 1))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay,clears", [("token", ()), ("slow", CLEARS), ("head", ())],
                         ids=["token", "clears", "head"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_attention_backward(shape, decay, clears, dtype):
    check_bwd(attn_inputs(*shape, dtype, seed=sum(shape) + 1, decay=decay, clears=clears,
                          h0=shape[1] % 2 == 1))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay", ["strong", "none"])
def test_attention_decay_extremes(decay, dtype):
    """Chunks whose whole decay underflows, and no decay at all."""
    x = attn_inputs(1, 300, 2, 2, 128, 64, dtype, seed=5, decay=decay, h0=True)
    check_fwd(x)
    check_bwd(x)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attention_every_token_clears(dtype):
    """Rows that see nothing but themselves: o_t = scale (q_t . k_t) v_t."""
    x = attn_inputs(1, 150, 2, 2, 64, 64, dtype, seed=6, clears=range(150), h0=True)
    o, hT = run_fwd(x)
    q, k, v = f64(x["q"]), f64(x["k"]), f64(x["v"])
    assert off(o, x["scale"] * np.sum(q * k, -1, keepdims=True) * v) <= TOL[dtype]
    assert off(hT, np.einsum("bhi,bhj->bhij", k[:, -1], v[:, -1])) <= STATE_TOL
    assert torch.all(run_bwd(x)["g"] == 0) and torch.all(run_bwd(x)["h0"] == 0)


def test_attention_many_heads_and_long_segments():
    """(batch, head)s that fill the GPU (no split), and few that are split."""
    for shape in ((3, 260, 64, 16, 128, 128), (1, 4500, 1, 1, 128, 128)):
        x = attn_inputs(*shape, BF, seed=7, decay="slow", clears=(100,))
        check_fwd(x)
        check_bwd(x)


def test_attention_gate_gradient_over_thousands_of_tokens():
    """One segment of 4096 tokens with memories of tens of tokens."""
    x = attn_inputs(1, 4096, 152, 152, 64, 64, BF, seed=8, decay="slow")
    got = run_bwd(x)["g"]
    pick = [0, 75, 151]
    sub = {n: (t[:, :, pick].contiguous() if torch.is_tensor(t) and t.dim() >= 3 else t)
           for n, t in x.items()}
    ref = attn_grad_oracle(sub)["g"]
    assert off(got[:, :, pick], ref) <= GATE_TOL


def test_attention_fixed_decays_with_memories_of_thousands_of_tokens():
    """Fixed decays close to 1 in fp32: a chunk's decay is the same all along, so its
    rounding must not add up over the ~90 chunks in memory. 2e-6: products kept to 2^-21,
    and one rounding of 2^-24 a chunk, 90 of them at random 6e-7."""
    x = attn_inputs(1, 6001, 8, 4, 64, 64, F32, seed=21, h0=True)
    x["g"] = -1.0 / torch.linspace(3000.0, 23000.0, 8, device="cuda")
    o, hT = run_fwd(x)
    ro, rh = attn_oracle(x)
    assert off(o, ro) <= 2e-6
    assert off(hT, rh) <= 2e-6


def test_attention_gradient_against_differences():
    """fp32, along a random direction: the loss's difference against <grad, d>. The
    second-order term (step^2) and the losses' rounding (1e-6 over the step) both
    stay under 1e-2 of the slope."""
    x = attn_inputs(1, 130, 2, 1, 64, 64, F32, seed=9, h0=True)
    loss = lambda y: sum(float((a.double() * b.double()).sum())  # noqa: E731
                         for a, b in zip(run_fwd(y), (x["dO"], x["dhT"])))
    got = run_bwd(x)
    for n in ("q", "k", "v", "g", "h0"):
        d = torch.randn_like(x[n])
        e = 2e-3
        num = (loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e)
        slope = float((got[n].double() * d.double()).sum())
        size = float(got[n].double().norm())
        assert abs(num - slope) <= 1e-2 * size, n


def test_attention_runs_are_identical():
    x = attn_inputs(1, 1500, 4, 2, 128, 128, BF, seed=10, h0=True)
    a, b = run_bwd(x), run_bwd(x)
    assert all(torch.equal(a[n], b[n]) for n in a)
    assert all(torch.equal(u, v) for u, v in zip(run_fwd(x), run_fwd(x)))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attention_takes_parts_of_a_projection(dtype):
    B, T, H, Hk, d = 2, 140, 4, 2, 64
    p = torch.randn(B, T, (2 * Hk + H) * d + 32, device="cuda").to(dtype)
    q, k = p[..., :Hk * d].unflatten(-1, (Hk, d)), p[..., Hk * d:2 * Hk * d].unflatten(-1, (Hk, d))
    v = p[..., 2 * Hk * d:(2 * Hk + H) * d].unflatten(-1, (H, d))
    g = -torch.rand(B, T, H, device="cuda")
    dO = torch.randn(B, T, H, d, device="cuda").to(dtype)
    a = gdr.decay_chunk_fwd(q, k, v, g)
    b = gdr.decay_chunk_fwd(q.contiguous(), k.contiguous(), v.contiguous(), g)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = gdr.decay_chunk_bwd(q, k, v, g, dO)
    b = gdr.decay_chunk_bwd(q.contiguous(), k.contiguous(), v.contiguous(), g, dO)
    assert all(torch.equal(a[n], b[n]) for n in a)
    state = torch.randn(B, H, d, d, device="cuda")
    s2 = state.clone()
    g3 = g[:, 3].contiguous()
    o1 = gdr.decay_step(q[:, 3], k[:, 3], v[:, 3], g3, state)
    o2 = gdr.decay_step(q[:, 3].contiguous(), k[:, 3].contiguous(), v[:, 3].contiguous(), g3, s2)
    assert torch.equal(o1, o2) and torch.equal(state, s2)


def test_attention_offsets_past_32_bits():
    """Tokens 60 million elements apart: the last ones lie past 2^31."""
    T, step = 40, 60_000_000
    base = torch.empty(T * step, dtype=BF, device="cuda")
    q, k, v = (base.as_strided((1, T, 1, 64), (T * step, step, 64, 1), at) for at in (0, 64, 128))
    x = attn_inputs(1, T, 1, 1, 64, 64, BF, seed=11)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        t.copy_(x[n])
    far = {**x, "q": q, "k": k, "v": v}
    assert all(torch.equal(a, b) for a, b in zip(run_fwd(far), run_fwd(x)))
    a, b = run_bwd(far), run_bwd(x)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_attention_in_place_state_and_other_stream():
    x = attn_inputs(1, 900, 2, 2, 128, 128, BF, seed=12, h0=True)
    o, hT = run_fwd(x)
    h = x["h0"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, h2 = gdr.decay_chunk_fwd(x["q"], x["k"], x["v"], x["g"], h, scale=x["scale"], hT=h,
                                 stream=side)
    grads = gdr.decay_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"], x["dhT"],
                                scale=x["scale"], stream=side)
    side.synchronize()
    assert h2 is h and torch.equal(o, o2) and torch.equal(hT, h)
    ref = run_bwd(x)
    assert all(torch.equal(ref[n], grads[n]) for n in ref)


def test_attention_prefix_ignores_a_later_chunk():
    """A NaN reaches no token of an earlier chunk."""
    x = attn_inputs(1, 300, 1, 1, 64, 64, BF, seed=13)
    o, _ = run_fwd(x)
    x["v"][0, 290] = torch.nan
    o2, h2 = run_fwd(x)
    assert torch.equal(o[:, :256], o2[:, :256])
    assert torch.isnan(o2[:, 290:]).all() and torch.isnan(h2).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,H,Hk,dk,dv,head", [(1, 1, 1, 64, 64, False), (3, 4, 2, 128, 64, True),
                                              (5, 2, 1, 64, 128, False),
                                              (40, 8, 8, 128, 128, False)])
def test_step(N, H, Hk, dk, dv, head, dtype):
    x = attn_inputs(N, 1, H, Hk, dk, dv, dtype, seed=N, decay="head" if head else "token", h0=True,
                    clears=(0,) if N == 5 else ())
    state = x["h0"].clone()
    o = gdr.decay_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0],
                       x["g"] if head else x["g"][:, 0], state, scale=x["scale"])
    torch.cuda.synchronize()
    ro, rh = attn_oracle(x)
    # one fused multiply-add per state element; a sum of d_k products and a rounding
    assert off(state, rh) <= 1e-6
    assert off(o, ro[:, 0]) <= (2e-6 if dtype == F32 else 2 ** -9)


def test_prefill_then_steps_is_one_prefill():
    x = attn_inputs(2, 70, 3, 3, 64, 128, F32, seed=14)
    o, hT = run_fwd(x)
    head = {n: (t[:, :60].contiguous() if n in "qkvg" else t) for n, t in x.items()}
    o1, state = run_fwd(head)
    outs = [o1] + [gdr.decay_step(x["q"][:, t], x["k"][:, t], x["v"][:, t], x["g"][:, t].contiguous(),
                                  state, scale=x["scale"])[:, None] for t in range(60, 70)]
    assert off(torch.cat(outs, 1), f64(o)) <= 2e-5 and off(state, f64(hT)) <= 2e-5


# ------------------------------------------------------------------ norm

NORM_SHAPES = [(1, 8), (3, 64), (37, 136), (5, 1000), (1, 2048), (700, 520), (33, 4096), (3, 8192)]


def norm_inputs(rows, D, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return r(rows, D).to(dtype), (3 * r(rows, D)).to(dtype), 1 + 0.1 * r(D)


def summed(x, res):
    return (x.float() + res.float()).to(x.dtype)


def near(got, ref, dtype, slack=4e-6):
    band = (2.0 ** -8 if dtype == BF else 2e-6) * np.abs(ref) + slack * np.abs(ref).max()
    assert (np.abs(f64(got) - ref) <= band).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,D", NORM_SHAPES)
def test_norm(rows, D, dtype):
    x, res, w = norm_inputs(rows, D, dtype, rows + D)
    y, r = gdr.add_rmsnorm(x, res, w, 1e-5)
    assert torch.equal(r, summed(x, res))
    near(y, layer.add_rmsnorm(f64(r), f64(w), 1e-5), dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,D", NORM_SHAPES)
def test_norm_to_8_bits(rows, D, dtype):
    x, res, w = norm_inputs(rows, D, dtype, rows + D)
    x[0] = -res[0]                        # a row of zeros: scale 1
    if D >= 136:
        w[:128] = 0.0                     # a block of zeros in every row
    y, s, r = gdr.add_rmsnorm_fp8(x, res, w, 1e-5)
    assert y.dtype == torch.float8_e4m3fn and s.shape == (rows, -(-D // 128))
    assert torch.equal(r, summed(x, res))
    ref = layer.add_rmsnorm(f64(r), f64(w), 1e-5)
    scale = layer.block_scales(ref)
    np.testing.assert_allclose(f64(s), scale, rtol=1e-6)
    assert torch.all(s[0] == 1) and torch.all(y[0].float() == 0)
    wide = np.repeat(scale, 128, axis=1)[:, :D]
    got = f64(y.float()) * np.repeat(f64(s), 128, axis=1)[:, :D]
    # half a step of a 3-bit mantissa, or of the smallest numbers
    band = 2.0 ** -4 * np.abs(ref) * (1 + 1e-4) + 2.0 ** -10 * wide * (1 + 1e-4)
    assert (np.abs(got - ref) <= band).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,D", NORM_SHAPES)
@pytest.mark.parametrize("with_res", [False, True])
def test_norm_gradients(rows, D, dtype, with_res):
    dy, r, w = norm_inputs(rows, D, dtype, rows + D + 1)
    dres = dy.flip(0).contiguous() if with_res else None
    dx, dw = gdr.add_rmsnorm_bwd(dy, r, w, 1e-5, dres=dres)
    rx, rw = layer.add_rmsnorm_gradients(f64(dy), f64(r), f64(w), 1e-5, f64(dres))
    near(dx, rx, dtype)
    assert off(dw, rw) <= 1e-5 if rows > 1 or D > 8 else True
    a, b = gdr.add_rmsnorm_bwd(dy, r, w, 1e-5, dres=dres), (dx, dw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_gradient_against_differences():
    """fp32: the slope along a random direction; step^2 and rounding over the step are
    both under 1e-2 of it."""
    dy, r, w = norm_inputs(6, 64, F32, 3)
    dx, dw = gdr.add_rmsnorm_bwd(dy, r, w, 1e-5)
    zero = torch.zeros_like(r)
    loss = lambda a, b: float((gdr.add_rmsnorm(a, zero, b, 1e-5)[0].double() * dy.double()).sum())  # noqa: E731
    e = 1e-2
    for grad, d, f in ((dx, torch.randn_like(r), lambda s, d: loss(r + s * d, w)),
                       (dw, torch.randn_like(w), lambda s, d: loss(r, w + s * d))):
        num = (f(e, d) - f(-e, d)) / (2 * e)
        assert abs(num - float((grad.double() * d.double()).sum())) <= 1e-2 * float(grad.norm())


def test_norm_in_place_empty_and_non_finite():
    x, res, w = norm_inputs(9, 256, BF, 4)
    y, r = gdr.add_rmsnorm(x, res, w)
    x2, res2 = x.clone(), res.clone()
    y2, r2 = gdr.add_rmsnorm(x2, res2, w, out=x2, residual_out=res2)
    assert y2 is x2 and r2 is res2 and torch.equal(y, y2) and torch.equal(r, r2)
    e = x[:0]
    assert gdr.add_rmsnorm(e, e, w)[0].shape == (0, 256)
    assert gdr.add_rmsnorm_fp8(e, e, w)[1].shape == (0, 2)
    assert torch.all(gdr.add_rmsnorm_bwd(e, e, w)[1] == 0)
    x[2, 200] = torch.nan
    x[4, 7] = torch.inf
    y3, s3, _ = gdr.add_rmsnorm_fp8(x, res, w)
    assert torch.isnan(y3[2].float()).all() and torch.isnan(s3[2]).all()
    assert torch.isnan(y3[4].float()[7])
    ok = [0, 1, 3, 5, 6, 7, 8]
    y4, s4, _ = gdr.add_rmsnorm_fp8(*norm_inputs(9, 256, BF, 4))
    assert torch.equal(y3.float()[ok], y4.float()[ok]) and torch.equal(s3[ok], s4[ok])


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,H,Hk,d,rot", [(1, 1, 1, 1, 16, 16), (7, 1, 32, 4, 128, 32),
                                           (2, 33, 3, 2, 64, 64), (1, 70, 5, 1, 80, 48)])
def test_rotary(B, T, H, Hk, d, rot, interleaved, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    q = torch.randn(B, T, H, d, generator=gen, device="cuda").to(dtype)
    k = torch.randn(B, T, Hk, d, generator=gen, device="cuda").to(dtype)
    cos, sin = gdr.rotary_table(5000, rot)
    pos = torch.randint(0, 5000, (B, T), generator=gen, device="cuda", dtype=torch.int32)
    for inverse in (False, True):
        a, b = gdr.rotary(q, k, cos, sin, pos, interleaved=interleaved, inverse=inverse)
        p = pos.long()
        c, s = f64(cos[p][:, :, None]), f64(sin[p][:, :, None]) * (-1 if inverse else 1)
        for got, x in ((a, q), (b, k)):
            ref = layer.rotary(f64(x), c, s, interleaved)
            # two products of magnitude up to |x|, one rounding (2^-8 of a bf16 value)
            band = (2.0 ** -8 if dtype == BF else 3e-7) * np.maximum(np.abs(ref), 1e-6) + 3e-7 * 8
            assert (np.abs(f64(got) - ref) <= band).all()
            assert torch.equal(got[..., rot:], x[..., rot:])
    q2, k2 = q.clone(), k.clone()
    gdr.rotary(q2, k2, cos, sin, pos, interleaved=interleaved, inverse=True, q_out=q2, k_out=k2)
    assert torch.equal(q2, a) and torch.equal(k2, b)


def test_rotary_default_positions_parts_and_bounds():
    B, T, H, d = 2, 20, 3, 64
    p = torch.randn(B, T, 5 * H * d, device="cuda").to(BF)
    q, k = (p[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in (1, 3))
    cos, sin = gdr.rotary_table(64, d)
    pos = (torch.arange(T, device="cuda") + 9).expand(B, T).to(torch.int32).contiguous()
    a = gdr.rotary(q, k, cos, sin, start=9)
    b = gdr.rotary(q.contiguous(), k.contiguous(), cos, sin, pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    before = p.clone()
    gdr.rotary(q, k, cos, sin, start=9, q_out=q, k_out=k)
    assert torch.equal(q, b[0]) and torch.equal(k, b[1])
    assert torch.equal(p[..., :H * d], before[..., :H * d])
    # positions outside the table: that token's pairs read NaN, no other
    pos[0, 4], pos[1, 7] = -1, 64
    c = gdr.rotary(b[0], b[1], cos, sin, pos)[0]
    bad = torch.isnan(c).all(-1).all(-1)
    assert bad[0, 4] and bad[1, 7] and int(bad.sum()) == 2 and int(torch.isnan(c).sum()) == 2 * H * d
    # an empty batch, and only one of q and k
    assert gdr.rotary(q[:0], k[:0], cos, sin)[0].shape == (0, T, H, d)
    only = gdr.rotary(q[:, :, :0].contiguous(), k.contiguous(), cos, sin)
    assert only[0].numel() == 0 and only[1].shape == k.shape


@pytest.mark.parametrize("kind", [None, "linear", "base", "ramp"])
def test_rotary_tables(kind):
    n, rot = 3000, 64
    kw = dict(scaling=kind, factor=4.0, original_length=1024) if kind else {}
    cos, sin = gdr.rotary_table(n, rot, 10000.0, **kw)
    f = layer.rotary_frequencies(rot, 10000.0, kind, 4.0, 1024)
    ang = np.arange(n)[:, None] * f
    m = 0.1 * np.log(4.0) + 1 if kind == "ramp" else 1.0
    # one rounding to fp32 of values up to 1.14, and the fp64 angles' few ulps
    assert np.abs(f64(cos) - m * np.cos(ang)).max() <= 1.3e-7
    assert np.abs(f64(sin) - m * np.sin(ang)).max() <= 1.3e-7


# ------------------------------------------------------------------ together

def test_retention_layer_prefill_and_steps():
    """A prompt in one prefill, and as a prefill followed by steps: the same outputs up
    to the bf16 of the paths between (each output a sum over roundings of 2^-9)."""
    net = RetentionLayer(256, 4, kv_heads=2, head_dim=64, max_len=512)
    x = torch.randn(2, 150, 256, device="cuda").to(BF)
    res = torch.randn(2, 150, 256, device="cuda").to(BF)
    y, r, state = net.prefill(x, res)
    y1, r1, st = net.prefill(x[:, :140].contiguous(), res[:, :140].contiguous())
    assert off(y1, f64(y[:, :140])) <= 2e-2
    for t in range(140, 150):
        yt, rt = net.step(x[:, t].contiguous(), res[:, t].contiguous(), st, t)
        assert off(yt, f64(y[:, t])) <= 2e-2 and torch.equal(rt, r[:, t])
    assert off(st, f64(state)) <= 2e-2


def test_retention_layer_mixer_gradients():
    net = RetentionLayer(64, 2, head_dim=64, max_len=256)
    q, k, v, dO = (torch.randn(1, 100, 2, 64, device="cuda") for _ in range(4))
    got = net.mixer_gradients(q, k, v, dO)
    f = lambda a, b, c: float((gdr.decay_chunk_fwd(  # noqa: E731
        *gdr.rotary(a, b, net.cos, net.sin), c, net.g)[0].double() * dO.double()).sum())
    for n, d, at in (("q", torch.randn_like(q), 0), ("k", torch.randn_like(k), 1),
                     ("v", torch.randn_like(v), 2)):
        # linear in each of q, k, v: only rounding is left of the difference
        args = [q, k, v]
        plus = f(*[a + d if i == at else a for i, a in enumerate(args)])
        num = plus - f(*args)
        assert abs(num - float((got[n].double() * d.double()).sum())) <= 1e-3 * abs(plus) + 1e-2
