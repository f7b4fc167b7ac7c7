"""Edges of the layer operators that need no GPU: their float64 oracle
(oracle/layer.py) and the wrappers' checks."""
import numpy as np
import pytest
import torch

from gated_delta_rule_10_gb300 import layer as wrappers
from oracle import layer

LONG = [(64, 65536), (64, 131072), (128, 131072), (128, 4096), (32, 2 ** 20)]


@pytest.mark.parametrize("rot,original", LONG)
def test_ramp_divides_in_full_only_what_turns_too_little(rot, original):
    """By the turns themselves: at least `fast` over the original length keeps a
    frequency, more than `slow` does not divide it in full (one channel's slack at each
    end, whose j is rounded outwards), and between the ends the share is linear in j."""
    factor, fast, slow, base = 4.0, 32.0, 1.0, 10000.0
    f = layer.rotary_frequencies(rot, base)
    r = layer.rotary_frequencies(rot, base, "ramp", factor, original, fast, slow)
    turns = original * f / (2 * np.pi)
    share = (1 - r / f) / (1 - 1 / factor)          # 0: kept, 1: divided in full
    step = base ** (2.0 / rot)                      # turns from one channel to the next
    assert np.all(share[turns >= fast * step] == 0)
    assert np.all(share[turns > slow] < 1 - 1e-9)
    np.testing.assert_allclose(share[turns < slow / step], 1.0, rtol=1e-12)
    on = share[(share > 1e-9) & (share < 1 - 1e-9)]
    np.testing.assert_allclose(np.diff(on, 2), 0.0, atol=1e-12)
    # its slope reaches from `fast` to `slow` turns, a channel more at each end at most
    span = np.log(fast / slow) / np.log(step)
    assert np.all(1 / np.diff(on) >= span - 1e-6) and np.all(1 / np.diff(on) <= span + 2 + 1e-6)


def test_ramp_by_hand():
    """rot 64, base 10000, 131072 positions: the last frequency turns 2.78 times; the ramp
    runs from channel 22 (22.51, of 32 turns) to 35 (34.55, of one), so that channel 31
    keeps 1 - (9 / 13) (3 / 4) of its own."""
    f = layer.rotary_frequencies(64, 10000.0)
    r = layer.rotary_frequencies(64, 10000.0, "ramp", 4.0, 131072)
    assert r[31] / f[31] == pytest.approx(1 - 9 / 13 * 0.75)


def test_a_workspace_elsewhere_is_refused():
    """A caller's workspace is written by the kernels: it has to be the device's."""
    dev = torch.device("cuda", 0)
    assert wrappers._workspace_bytes(None, dev) == 0
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        wrappers._workspace_bytes(torch.empty(4096, dtype=torch.uint8), dev)
