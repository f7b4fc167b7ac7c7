"""GPU tests of the block operators at the edges of what their header allows, against the float64
oracle. Bars as in test_block_gpu.py, or derived at the test."""
import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from oracle import block
from test_block_gpu import BF, DTYPES, f64, near, norms_inputs, off, rnd

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
