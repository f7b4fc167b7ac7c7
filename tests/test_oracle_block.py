"""The block operators' float64 oracle: against torch's autograd on the same formulas, and
by hand."""
import numpy as np
import pytest
import torch

from oracle import block


def leaf(*arrays):
    return [None if a is None else torch.tensor(a, dtype=torch.float64, requires_grad=True)
            for a in arrays]


def same(got, ref):
    np.testing.assert_allclose(got, ref.detach().numpy() if torch.is_tensor(ref) else ref,
                               rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("T,K", [(1, 4), (2, 4), (9, 3), (6, 2)])
@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("packed", [True, False])
def test_short_conv(T, K, act, packed):
    rng = np.random.default_rng(T + K)
    D = 5
    x, w, b, s0 = (rng.standard_normal(n) for n in ((T, D), (D, K), D, (K - 1, D)))
    dy, dl = rng.standard_normal((T, D)), rng.standard_normal((K - 1, D))
    starts = (rng.random(T) < 0.3) if packed else None
    y, last = block.short_conv(x, w, b, s0, starts, act)
    tx, tw, tb, ts = leaf(x, w, b, s0)
    rows = torch.cat([ts, tx])
    out, ends = [], []
    for t in range(T):
        s = tb
        for j in range(K):            # j tokens back, if no document starts in between
            if starts is None or not starts[max(t - j + 1, 0):t + 1].any():
                s = s + tw[:, K - 1 - j] * rows[K - 1 + t - j]
        out.append(torch.nn.functional.silu(s) if act else s)
    for i in range(K - 1):
        t = T - (K - 1) + i
        cut = starts is not None and starts[max(t + 1, 0):].any()
        ends.append(torch.zeros(D, dtype=torch.float64) if cut else rows[K - 1 + t])
    ty, tl = torch.stack(out), torch.stack(ends)
    same(y, ty)
    same(last, tl)
    loss = (ty * torch.tensor(dy)).sum() + (tl * torch.tensor(dl)).sum()
    grads = torch.autograd.grad(loss, (tx, tw, tb, ts), allow_unused=True)
    got = block.short_conv_gradients(dy, x, w, b, s0, dl, starts, act)
    for n, g, like in zip(("x", "weight", "bias", "state"), grads, (x, w, b, s0)):
        same(got[n], np.zeros_like(like) if g is None else g)


@pytest.mark.parametrize("T,G,plus,gated,packed", [(1, 1, True, True, False), (7, 2, True, True, True),
                                                   (7, 1, False, False, False),
                                                   (5, 3, True, False, True)])
def test_state_space(T, G, plus, gated, packed):
    rng = np.random.default_rng(T + G)
    D, N = 6, 4
    r = rng.standard_normal
    x, dt, B, C, h0, skip, bias = (r(n) for n in ((T, D), (T, D), (T, G, N), (T, G, N), (D, N), D, D))
    A = -np.exp(r((D, N)))
    z = r((T, D)) if gated else None
    if not plus:
        dt, bias = 0.1 * dt, 0.1 * bias
    starts = (rng.random(T) < 0.4) if packed else None
    dy, dhT = r((T, D)), r((D, N))
    y, h = block.state_space(x, dt, A, B, C, h0, skip, z, bias, plus, starts)
    tx, tdt, tA, tB, tC, th, ts, tz, tb = leaf(x, dt, A, B, C, h0, skip, z, bias)
    u = tdt + tb
    if plus:
        u = torch.nn.functional.softplus(u)
    s, out = th, []
    for t in range(T):
        wide = lambda v: v[t].repeat_interleave(D // G, 0)  # noqa: E731
        if starts is not None and starts[t]:
            s = torch.zeros_like(s)
        s = torch.exp(u[t][:, None] * tA) * s + (u[t] * tx[t])[:, None] * wide(tB)
        o = (s * wide(tC)).sum(1) + ts * tx[t]
        out.append(o if z is None else o * torch.nn.functional.silu(tz[t]))
    ty = torch.stack(out)
    same(y, ty)
    same(h[-1], s)
    leaves = {"x": tx, "dt": tdt, "A": tA, "B": tB, "C": tC, "h0": th, "skip": ts, "dt_bias": tb}
    if gated:
        leaves["z"] = tz
    loss = (ty * torch.tensor(dy)).sum() + (s * torch.tensor(dhT)).sum()
    grads = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    got = block.state_space_gradients(dy, x, dt, A, B, C, h0, dhT, skip, z, bias, plus, starts)
    for (n, like), g in zip(leaves.items(), grads):
        same(got[n], np.zeros(like.shape) if g is None else g)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("scaled", [True, False])
def test_block_norms(gated, scaled):
    rng = np.random.default_rng(3)
    r = rng.standard_normal
    x, res, dy, dres = (r((4, 10)) for _ in range(4))
    post, pre = r(10), r(10)
    gate, scale = (r((4, 10)) if gated else None), (r(10) if scaled else None)
    total = block.block_sum(x, res, post, gate, scale)
    tx, tr, tp, tq, tg, ts = leaf(x, res, post, pre, gate, scale)
    norm = lambda v, w: v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    u = norm(tx, tp)
    u = u * ts if scaled else u
    u = u * torch.sigmoid(tg) if gated else u
    ta = tr + u
    same(total, ta)
    same(block.pre_norm(total, pre), norm(ta, tq))
    leaves = {"x": tx, "residual": tr, "post": tp, "pre": tq}
    if gated:
        leaves["gate"] = tg
    if scaled:
        leaves["scale"] = ts
    loss = (norm(ta, tq) * torch.tensor(dy)).sum() + (ta * torch.tensor(dres)).sum()
    grads = torch.autograd.grad(loss, list(leaves.values()))
    got = block.block_norms_gradients(dy, x, total, post, pre, gate, scale, dres)
    for n, g in zip(leaves, grads):
        same(got[n], g)


def test_by_hand():
    """Two taps over 1, 2, 4 with a document's start at the last: 3 * 1, 3 * 2 + 5 * 1, 3 * 4.
    One channel and state, u = 1, A = -ln 2: 1, 1/2 + 2, 4 (cleared)."""
    y, last = block.short_conv(np.array([[1.0], [2.0], [4.0]]), np.array([[5.0, 3.0]]),
                               starts=np.array([0, 0, 1]), act=False)
    np.testing.assert_allclose(y[:, 0], [3.0, 11.0, 12.0])
    np.testing.assert_allclose(last, [[4.0]])
    one = np.ones((3, 1))
    y, h = block.state_space(np.array([[1.0], [2.0], [4.0]]), one, np.array([[-np.log(2.0)]]),
                             one[:, None], one[:, None], plus=False, starts=np.array([0, 0, 1]))
    np.testing.assert_allclose(y[:, 0], [1.0, 2.5, 4.0])
