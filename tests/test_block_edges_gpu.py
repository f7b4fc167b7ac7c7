"""GPU tests of the block operators at the edges of what their header allows, against the float64
oracle. Bars as in test_block_gpu.py, or derived at the test."""
import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from oracle import block
from test_block_gpu import DTYPES, f64, near, norms_inputs, off, rnd

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
