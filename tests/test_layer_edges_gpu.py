"""Edges of the layer operators on the GPU, against the float64 oracle
(oracle/layer.py); the bars are those of test_layer_gpu.py unless a test says its own."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from gated_delta_rule_10_gb300 import layer as wrappers
from oracle import layer
from test_layer_gpu import (BF, F32, GATE_TOL, STATE_TOL, TOL, attn_grad_oracle, attn_inputs,
                            attn_oracle, check_bwd, check_fwd, f64, near, norm_inputs, off,
                            run_bwd, run_fwd)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ linear attention

def backward_call(x, dhT, dh0):
    """gdr_decay_chunk_bwd through the C ABI: dh0 (a tensor, or None) is the caller's."""
    B, T, H, dv = x["v"].shape
    Hk, dk = x["q"].shape[2:]
    dt = x["q"].dtype
    s = wrappers.DecayShape(B, T, H, Hk, dk, dv, gdr.GDR_BF16 if dt == BF else gdr.GDR_F32,
                            int(x["g"].dim() == 1), x["scale"], 0, 0, 0)
    out = {"q": torch.empty_like(x["q"]), "k": torch.empty_like(x["k"]),
           "v": torch.empty_like(x["v"]), "g": torch.empty_like(x["g"])}
    ws = torch.empty(gdr.decay_chunk_bwd_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = wrappers._lib().gdr_decay_chunk_bwd(
        ctypes.byref(s), *(p(x[n]) for n in ("q", "k", "v", "g", "h0", "dO")), p(dhT),
        *(p(out[n]) for n in ("q", "k", "v", "g")), p(dh0), p(ws), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 100, 3, 1, 64, 128), (3, 520, 64, 32, 128, 128),
                                   (1, 1300, 2, 2, 128, 64)], ids=lambda s: "x".join(map(str, s)))
def test_backward_with_the_state_gradients_in_one_buffer(shape, dtype):
    """dhT and dh0 may be one buffer: the same bits as with two, uncut (one chunk, and
    several with more (batch, head)s than SMs) and cut into segments."""
    x = attn_inputs(*shape, dtype, seed=51, h0=True)
    ref = run_bwd(x)
    for _ in range(3):
        both = x["dhT"].clone()
        got = backward_call(x, both, both)
        assert all(torch.equal(got[n], ref[n]) for n in got)
        assert torch.equal(both, ref["h0"])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape,decay", [((1, 900, 2, 1, 64, 128), "slow"),
                                         ((2, 130, 80, 40, 128, 64), "head"),
                                         ((1, 200, 3, 3, 128, 128), "token")],
                         ids=lambda c: c if isinstance(c, str) else "x".join(map(str, c)))
def test_backward_without_the_state_gradient(shape, decay, dtype):
    """The other gradients are the same bits whether or not that of h0 is asked for."""
    x = attn_inputs(*shape, dtype, seed=52, decay=decay, h0=True)
    ref = run_bwd(x)
    got = backward_call(x, x["dhT"], None)
    assert all(torch.equal(got[n], ref[n]) for n in got)


@pytest.mark.parametrize("decay", ["slow", "fixed"])
def test_gate_gradient_from_a_state_over_thousands_of_tokens(decay):
    """One segment of 4096 tokens that starts from a state, as does the gate's gradient."""
    x = attn_inputs(1, 4096, 152, 152, 64, 64, BF, seed=53, decay="slow", h0=True)
    if decay == "fixed":
        x["g"] = -1.0 / torch.linspace(2.0, 20000.0, 152, device="cuda")
    got, pick = run_bwd(x)["g"], [0, 75, 151]
    sub = {n: t[:, pick] if n in ("h0", "dhT") else t[..., pick] if n == "g" else t[:, :, pick]
           if torch.is_tensor(t) else t for n, t in x.items()}
    assert off(got[..., pick], attn_grad_oracle(sub)["g"]) <= GATE_TOL


def pieces(x, backward):
    """The pieces of each sequence whose own states are computed, from the workspace's size:
    the states are [B * H, pieces (backward: + 1, and twice), dk, dv] fp32, and everything
    else but the backward's terms by token takes less than one more of them."""
    B, T, H, dv = x["v"].shape
    Hk, dk = x["q"].shape[2:]
    bf = x["q"].dtype == BF
    s = wrappers.DecayShape(B, T, H, Hk, dk, dv, gdr.GDR_BF16 if bf else gdr.GDR_F32,
                            int(x["g"].dim() == 1), x["scale"], 0, 0, 0)
    states = 4 * B * H * dk * dv
    if not backward:
        return gdr.decay_chunk_fwd_workspace_bytes(s) // states
    planes = 2 * (dk // 64 + 1) + 2 if bf else 5
    terms = 4 * B * H * T * (planes + (2 * dk if Hk != H else 0))
    return (gdr.decay_chunk_bwd_workspace_bytes(s) - terms) // (2 * states) - 1


def heads_of(x, pick):
    """Those heads alone (q and k of their own)."""
    r = x["v"].shape[2] // x["q"].shape[2]
    at = {"q": [h // r for h in pick], "k": [h // r for h in pick]}
    return {n: t if not torch.is_tensor(t) else t[:, pick] if n in ("h0", "dhT")
            else t[..., pick] if n == "g" else t[:, :, at.get(n, pick)] for n, t in x.items()}


def check_heads(x, pick):
    """check_fwd and check_bwd, of some heads; dq and dk where they are not shared."""
    dt, sub = x["q"].dtype, heads_of(x, pick)
    o, hT = run_fwd(x)
    ro, rh = attn_oracle(sub)
    assert off(o[:, :, pick], ro) <= TOL[dt]
    assert off(hT[:, pick], rh) <= STATE_TOL
    got, ref = run_bwd(x), attn_grad_oracle(sub)
    for n in ("v",) if x["q"].shape[2] != x["v"].shape[2] else ("q", "k", "v"):
        assert off(got[n][:, :, pick], ref[n]) <= TOL[dt], n
    assert off(got["h0"][:, pick], ref["h0"]) <= STATE_TOL
    assert off(got["g"][..., pick], ref["g"]) <= GATE_TOL


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay,clears", [("slow", ()), ("slow", (100, 511, 512, 640)), ("head", ())],
                         ids=["slow", "clears", "head"])
@pytest.mark.parametrize("shape", [(1, 1101, 3, 1, 64, 128), (2, 1090, 2, 2, 128, 64),
                                   (1, 2050, 1, 1, 128, 128)], ids=lambda s: "x".join(map(str, s)))
def test_segments_from_a_state(shape, decay, clears, dtype):
    """Sequences cut into segments, from a given state and with a given gradient of the
    last one."""
    x = attn_inputs(*shape, dtype, seed=56, decay=decay, clears=clears, h0=True)
    assert pieces(x, False) >= 2 and pieces(x, True) >= 2
    check_fwd(x)
    check_bwd(x)


@pytest.mark.parametrize("states", [True, False], ids=["states", "zero"])
@pytest.mark.parametrize("decay", ["slow", "head"])
@pytest.mark.parametrize("dtype,T,H,Hk,backward", [(BF, 2100, 32, 32, True), (BF, 2100, 32, 8, True),
                                                   (F32, 300, 64, 64, False),
                                                   (F32, 300, 32, 32, True)])
def test_segments_of_several_pieces(dtype, T, H, Hk, backward, decay, states):
    """Segments whose own states are computed in several pieces: more pieces than there are
    segments, of which no more than fill 152 SMs are made (a CTA each for the forward, for
    64 columns of bf16; two in the fp32 backward)."""
    x = attn_inputs(1, T, H, Hk, 128, 128, dtype, seed=57, decay=decay, h0=states)
    ctas = H * (2 if dtype == BF or backward else 1)
    assert pieces(x, backward) > 152 // ctas >= 2
    check_heads(x, [0, H // 2 + 1, H - 1])


def test_a_training_batch():
    """4 x 4096 x 16 heads x 128: one head of each sequence."""
    x = attn_inputs(4, 4096, 16, 16, 128, 128, BF, seed=59, decay="slow", clears=(700, 2800))
    check_heads(x, [11])


def test_segments_of_a_long_backward_that_fills_the_gpu():
    """More (batch, head)s than SMs: the forward runs uncut, the backward's segments end
    after 4096 tokens all the same."""
    x = attn_inputs(1, 4400, 160, 160, 64, 64, BF, seed=58, decay="slow", h0=True)
    assert pieces(x, False) == 0 and pieces(x, True) >= 2
    check_heads(x, [0, 79, 159])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gate_gradient_of_fixed_decays_with_a_gradient_of_the_last_state(dtype):
    """The last state's gradient is felt in the last tokens; what is rounded there must not
    add up over the 4096 whose sum a fixed decay's gradient is."""
    x = attn_inputs(1, 4096, 32, 32, 128, 128, dtype, seed=57, decay="head", h0=True)
    pick = [0, 17, 31]
    ref = attn_grad_oracle(heads_of(x, pick))["g"]
    assert off(run_bwd(x)["g"][pick], ref) <= GATE_TOL


def test_callers_workspaces():
    """Large enough, of any type: the same bits; elsewhere, or with gaps: refused before
    any launch, and too small by the library."""
    x = attn_inputs(1, 700, 2, 1, 64, 64, BF, seed=54, h0=True)
    dy, w = torch.randn(40, 256, device="cuda"), torch.ones(256, device="cuda")
    y = attn_inputs(1, 1500, 2, 1, 64, 64, BF, seed=55)
    calls = [lambda **k: gdr.decay_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], **k),   # none needed
             lambda **k: gdr.decay_chunk_fwd(y["q"], y["k"], y["v"], y["g"], **k),
             lambda **k: tuple(gdr.decay_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["dO"], x["h0"],
                                                   x["dhT"], **k).values()),
             lambda **k: gdr.add_rmsnorm_bwd(dy, dy, w, **k)]
    n = 1 << 24
    for call in calls:
        for ws in (torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(n // 4, device="cuda")):
            assert all(torch.equal(a, b) for a, b in zip(call(), call(workspace=ws)))
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=torch.empty(n, dtype=torch.uint8))
        with pytest.raises(ValueError, match="contiguous"):
            call(workspace=torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2])
        if call is calls[0]:
            continue
        with pytest.raises(gdr.GdrError):
            call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("low,share", [(-103.9, 0.5), (-100.0, 0.1), (-60.0, 0.5), (-20.0, 0.5)])
def test_attention_decays_that_all_but_clear(low, share, dtype):
    """Tokens just above the clearing decay among slow ones: the sums of the log-decays
    reach thousands, and the pairs between those tokens still decay by their own."""
    x = attn_inputs(1, 300, 2, 2, 64, 128, dtype, seed=61, decay="slow", h0=True)
    gen = torch.Generator(device="cuda").manual_seed(62)
    at = torch.rand(1, 300, 2, generator=gen, device="cuda") < share
    x["g"] = torch.where(at, torch.full_like(x["g"], low), x["g"] / 100)
    check_fwd(x)
    check_bwd(x)


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("D", [64, 256, 1000, 4096])
def test_norm_to_8_bits_of_subnormal_blocks(D):
    """Blocks whose max / 448 is subnormal, or zero to the nearest."""
    x = torch.zeros(8, D, device="cuda")
    for i, m in enumerate((1e-45, 3e-45, 2e-44, 1e-43, 9e-43, 1e-41, 1e-39, 1e-36)):
        x[i, ::3] = m
        x[i, 1::3] = -m / 3
    w = torch.full((D,), 2.0 ** -10, device="cuda")
    y, s, _ = gdr.add_rmsnorm_fp8(x, torch.zeros_like(x), w, 1e-6)
    got = f64(y.float()) * np.repeat(f64(s), 128, axis=1)[:, :D]
    ref = layer.add_rmsnorm(f64(x), f64(w), 1e-6)
    # y is rounded to the subnormals' unit (a block that is then zero has scale 1); then
    # half a step of a 3-bit mantissa, or of the smallest 8-bit numbers at the scale
    unit = 2.0 ** -149
    wide = np.maximum(layer.block_scales(ref) * (layer.block_scales(ref) < 1), 2.0 ** -126)
    band = (2.0 ** -4 * (np.abs(ref) + unit) + 2.0 ** -10 * np.repeat(wide, 128, axis=1)[:, :D]) * \
        (1 + 1e-4) + unit
    assert (np.abs(got - ref) <= band).all()
    assert (f64(s) >= 2.0 ** -126).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_norm_of_rows_that_are_not_finite_or_overflow(dtype):
    """NaN: the whole row. Infinity: NaN there (in 8 bits in its block), zeros elsewhere.
    Finite values whose squares add up past fp32: zeros."""
    D = 400
    x, res, w = norm_inputs(5, D, dtype, 71)
    x[1, 200], x[2, 200], x[3, 7] = torch.nan, torch.inf, 3e19
    y, r = gdr.add_rmsnorm(x, res, w)
    y8, s, r8 = gdr.add_rmsnorm_fp8(x, res, w)
    assert torch.equal(r.isnan(), r8.isnan()) and torch.equal(r[2:], r8[2:])
    a, b, c = f64(y), f64(y8.float()), f64(s)
    assert np.isnan(a[1]).all() and np.isnan(b[1]).all() and np.isnan(c[1]).all()
    other = np.arange(D) != 200
    assert np.isnan(a[2, 200]) and (a[2, other] == 0).all()
    block = np.arange(D) // 128 == 1
    assert np.isnan(b[2, block]).all() and (b[2, ~block] == 0).all()
    assert np.isnan(c[2, 1]) and (c[2, [0, 2, 3]] == 1).all()
    assert (a[3] == 0).all() and (b[3] == 0).all() and (c[3] == 1).all()
    near(y[[0, 4]], layer.add_rmsnorm(f64(r[[0, 4]]), f64(w), 1e-6), dtype)


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("rot,original", [(64, 65536), (64, 131072), (128, 131072)])
def test_rotary_table_ramp_of_long_contexts(rot, original):
    """A ramp that ends past the last frequency."""
    n = 3000
    cos, sin = gdr.rotary_table(n, rot, 10000.0, scaling="ramp", factor=4.0,
                                original_length=original)
    ang = np.arange(n)[:, None] * layer.rotary_frequencies(rot, 10000.0, "ramp", 4.0, original)
    m = 0.1 * np.log(4.0) + 1
    # one rounding to fp32 of values up to 1.14, and the fp64 angles' few ulps
    assert np.abs(f64(cos) - m * np.cos(ang)).max() <= 1.3e-7
    assert np.abs(f64(sin) - m * np.sin(ang)).max() <= 1.3e-7
