"""Pins of the layer operators' float64 oracle (oracle/layer.py): worked values,
reductions, and gradients against central differences."""
import numpy as np
import pytest

from oracle import layer, recurrence

RNG = np.random.default_rng


def test_decay_recurrence_by_hand():
    # two tokens of width one: S = 2 * 3 = 6, then 6 / 2 + 5 * 7 = 38
    one = lambda *x: np.array(x, dtype=np.float64)[:, None]  # noqa: E731
    o, S = layer.decay_recurrence(one(1, 10), one(2, 5), one(3, 7), np.log([1.0, 0.5]))
    assert S[1, 0, 0] == 6 and S[2, 0, 0] == pytest.approx(38)
    assert o[:, 0] == pytest.approx([6, 380])


def test_decay_recurrence_is_the_masked_sum():
    r = RNG(0)
    T, dk, dv = 9, 4, 3
    q, k, v = r.normal(size=(T, dk)), r.normal(size=(T, dk)), r.normal(size=(T, dv))
    g = -np.abs(r.normal(size=T))
    o, _ = layer.decay_recurrence(q, k, v, g, scale=0.3)
    G = np.cumsum(g)
    for t in range(T):
        want = sum(np.exp(G[t] - G[i]) * (q[t] @ k[i]) * v[i] for i in range(t + 1))
        assert o[t] == pytest.approx(0.3 * want)


def test_decay_recurrence_is_the_delta_rule_without_the_erase():
    r = RNG(1)
    T, dk, dv = 7, 4, 4
    q, k, v = r.normal(size=(T, dk)), r.normal(size=(T, dk)), r.normal(size=(T, dv))
    g = -np.abs(r.normal(size=T))
    o, S = layer.decay_recurrence(q, k, v, g)
    # erase gate 0, write gate 1 in the general form
    o2, S2 = recurrence.unified(q, k, v, g, b=np.zeros((T, dk)), w=np.ones((T, dv)), scale=1.0,
                                flags=2 | 4)[:2]
    np.testing.assert_allclose(o, o2, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S[-1], S2, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("clears", [(), (0,), (3, 4)])
def test_decay_gradients_against_differences(clears):
    r = RNG(2)
    T, dk, dv = 7, 3, 4
    x = {"q": r.normal(size=(T, dk)), "k": r.normal(size=(T, dk)), "v": r.normal(size=(T, dv)),
         "g": -np.abs(r.normal(size=T)), "h0": r.normal(size=(dk, dv))}
    for t in clears:
        x["g"][t] = -np.inf
    dO, dhT = r.normal(size=(T, dv)), r.normal(size=(dk, dv))

    def loss(y):
        o, S = layer.decay_recurrence(y["q"], y["k"], y["v"], y["g"], y["h0"], scale=0.7)
        return np.sum(dO * o) + np.sum(dhT * S[-1])

    got = layer.decay_gradients(x["q"], x["k"], x["v"], x["g"], dO, x["h0"], dhT, scale=0.7)
    for n in x:
        d = r.normal(size=x[n].shape)
        if n == "g":
            d[list(clears)] = 0
            assert all(got["g"][t] == 0 for t in clears)
        e = 1e-6
        step = np.where(np.isinf(x[n]), 0.0, d * e)
        num = (loss({**x, n: x[n] + step}) - loss({**x, n: x[n] - step})) / (2 * e)
        assert num == pytest.approx(np.sum(got[n] * d), rel=1e-6, abs=1e-7), n


def test_norm_gradients_against_differences():
    r = RNG(3)
    x, w, dy, dres = (r.normal(size=s) for s in ((4, 6), (6,), (4, 6), (4, 6)))
    dx, dw = layer.add_rmsnorm_gradients(dy, x, w, 1e-3, dres)
    for arr, grad, f in ((x, dx, lambda y: np.sum(dy * layer.add_rmsnorm(y, w, 1e-3)) +
                          np.sum(dres * y)),
                         (w, dw, lambda y: np.sum(dy * layer.add_rmsnorm(x, y, 1e-3)))):
        d = r.normal(size=arr.shape)
        num = (f(arr + 1e-6 * d) - f(arr - 1e-6 * d)) / 2e-6
        assert num == pytest.approx(np.sum(grad * d), rel=1e-7)


def test_norm_by_hand():
    # mean of squares of (3, 4) is 12.5; scales of a block are max / 448
    y = layer.add_rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert y[0] == pytest.approx([3 / np.sqrt(12.5), 8 / np.sqrt(12.5)])
    z = np.zeros((1, 200))
    z[0, 5], z[0, 150] = -896.0, 0.0
    assert layer.block_scales(z).tolist() == [[2.0, 1.0]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_turns_and_turns_back(interleaved):
    r = RNG(4)
    x = r.normal(size=(5, 16))
    ang = r.normal(size=(5, 4))
    y = layer.rotary(x, np.cos(ang), np.sin(ang), interleaved)
    assert np.array_equal(y[:, 8:], x[:, 8:])
    assert np.linalg.norm(y, axis=1) == pytest.approx(np.linalg.norm(x, axis=1))
    np.testing.assert_allclose(layer.rotary(y, np.cos(ang), -np.sin(ang), interleaved), x,
                               atol=1e-14)


def test_rotary_pairs():
    x = np.arange(8.0)[None]
    c, s = np.zeros((1, 2)), np.ones((1, 2))       # a quarter turn of the first four
    assert layer.rotary(x, c, s, False)[0].tolist() == [-2, -3, 0, 1, 4, 5, 6, 7]
    assert layer.rotary(x, c, s, True)[0].tolist() == [-1, 0, -3, 2, 4, 5, 6, 7]


def test_rotary_frequencies_of_longer_contexts():
    f = layer.rotary_frequencies(64, 10000.0)
    assert f[0] == 1.0 and f[-1] == pytest.approx(10000.0 ** (-62 / 64))
    np.testing.assert_allclose(layer.rotary_frequencies(64, 1e4, "linear", 4.0), f / 4)
    b = layer.rotary_frequencies(64, 1e4, "base", 4.0)
    assert b[0] == 1.0 and b[-1] == pytest.approx(f[-1] / 4)
    r = layer.rotary_frequencies(64, 1e4, "ramp", 4.0, 4096)
    assert r[0] == f[0] and r[-1] == pytest.approx(f[-1] / 4)
    assert np.all(r <= f + 1e-15) and np.all(r >= f / 4 - 1e-15)
