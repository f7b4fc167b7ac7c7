"""Float64 oracle of the layer operators: linear attention with a decay for each
head (token recurrence and its gradients), the residual RMS norm (also to 8 bits
with scales) and rotary positions. Plain numpy loops over tokens, written from the
formulas; test infrastructure only.
"""
import numpy as np


def decay_recurrence(q, k, v, g, h0=None, scale=1.0):
    """S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t for one head.

    q, k [T, dk]; v [T, dv]; g [T]; h0 [dk, dv]. Returns o [T, dv] and all states
    [T + 1, dk, dv] (entry 0 is the start)."""
    T, dk = q.shape
    dv = v.shape[1]
    S = np.zeros((T + 1, dk, dv))
    if h0 is not None:
        S[0] = h0
    o = np.zeros((T, dv))
    for t in range(T):
        S[t + 1] = np.exp(g[t]) * S[t] + np.outer(k[t], v[t])
        o[t] = scale * (q[t] @ S[t + 1])
    return o, S


def decay_gradients(q, k, v, g, dO, h0=None, dhT=None, scale=1.0):
    """Gradients of <dO, o> + <dhT, S_T> by walking the recurrence backward."""
    _, S = decay_recurrence(q, k, v, g, h0, scale)
    T = q.shape[0]
    D = np.zeros_like(S[0]) if dhT is None else np.array(dhT, dtype=np.float64)
    dq, dk, dv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros(T)
    for t in range(T - 1, -1, -1):
        D = D + scale * np.outer(q[t], dO[t])       # the read-out of S_t
        dq[t] = scale * (S[t + 1] @ dO[t])
        dk[t] = D @ v[t]
        dv[t] = k[t] @ D
        a = np.exp(g[t])
        dg[t] = a * np.sum(D * S[t])
        D = a * D
    return {"q": dq, "k": dk, "v": dv, "g": dg, "h0": D}


def heads(fn, q, k, v, g, *rest, **kw):
    """Runs `fn` for every batch row and head: q, k [B,T,Hk,dk], v [B,T,H,dv], g
    [B,T,H]; entries of `rest` are [B,T,H,d], [B,H,dk,dv] or None. Yields (b, h,
    result)."""
    B, T, H, _ = v.shape
    r = H // q.shape[2]
    for b in range(B):
        for h in range(H):
            more = [None if x is None else (x[b, :, h] if x.shape[1] == T and x.shape[2] == H
                                            else x[b, h]) for x in rest]
            yield b, h, fn(q[b, :, h // r], k[b, :, h // r], v[b, :, h], g[b, :, h], *more, **kw)


def add_rmsnorm(r, weight, eps):
    """r / sqrt(mean r^2 + eps) * weight over the last axis."""
    return r / np.sqrt(np.mean(r * r, axis=-1, keepdims=True) + eps) * weight


def add_rmsnorm_gradients(dy, r, weight, eps, dres=None):
    rms = np.sqrt(np.mean(r * r, axis=-1, keepdims=True) + eps)
    n = r / rms
    dn = dy * weight
    dx = (dn - n * np.mean(dn * n, axis=-1, keepdims=True)) / rms
    return dx if dres is None else dx + dres, np.sum(dy * n, axis=0)


def block_scales(y):
    """max |y| / 448 of each 128 columns, 1 for a block of zeros."""
    out = []
    for c in range(0, y.shape[-1], 128):
        m = np.abs(y[..., c:c + 128]).max(axis=-1)
        out.append(np.where(m > 0, m / 448.0, 1.0))
    return np.stack(out, axis=-1)


def rotary(x, cos, sin, interleaved):
    """The pairs of the first 2 * cos.shape[-1] channels turned; x [..., d], cos and
    sin broadcastable to [..., rot / 2]."""
    half = cos.shape[-1]
    y = x.copy()
    a, b = ((x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved
            else (x[..., :half], x[..., half:2 * half]))
    u, v = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = u, v
    else:
        y[..., :half], y[..., half:2 * half] = u, v
    return y


def rotary_frequencies(rot, base, kind=None, factor=1.0, original=0, fast=32.0, slow=1.0):
    j = np.arange(rot // 2, dtype=np.float64)
    if kind == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * j / rot)
    if kind == "linear":
        f = f / factor
    if kind == "ramp":
        # the j at which a frequency turns r times over `original` positions
        at = lambda r: rot * np.log(original / (2 * np.pi * r)) / (2 * np.log(base))  # noqa: E731
        # ends outwards to whole j, within 0 and rot - 1 (the YaRN paper's bounds: the ramp
        # may end past the last frequency, rot / 2 - 1)
        lo, hi = max(np.floor(at(fast)), 0.0), min(np.ceil(at(slow)), rot - 1.0)
        r = np.clip((j - lo) / (hi - lo if hi > lo else 1e-3), 0.0, 1.0)
        f = f * (1 - r) + f / factor * r
    return f
