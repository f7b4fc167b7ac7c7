"""GPU tests of the block operators at the edges of what their header allows, against the float64
oracle. Bars as in test_block_gpu.py, or derived at the test."""
import pytest

import gated_delta_rule_10_gb300 as gdr
from oracle import block
from test_block_gpu import DTYPES, f64, near, norms_inputs, off

pytestmark = pytest.mark.gpu


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
