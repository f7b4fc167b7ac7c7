"""Edges of the layer operators on the GPU, against the float64 oracle
(oracle/layer.py); the bars are those of test_layer_gpu.py unless a test says its own."""
import numpy as np
import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from oracle import layer
from test_layer_gpu import f64

pytestmark = pytest.mark.gpu


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
