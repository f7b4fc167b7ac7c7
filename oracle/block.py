"""Float64 oracle of the block operators: the short causal convolution, the state space
recurrence and the norms after and before a block, with their gradients. Plain numpy loops
over tokens, written from the formulas; test infrastructure only.
"""
import numpy as np


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


def silu(x):
    return x * sigmoid(x)


def silu_slope(x):
    s = sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


def softplus(x):
    return np.logaddexp(0.0, x)


# ------------------------------------------------------------------ short convolution

def _documents(starts, K):
    """Number of the document of each row, state rows first (document 0)."""
    return np.concatenate([np.zeros(K - 1, int), np.cumsum(starts != 0)])


def short_conv(x, weight, bias=None, state=None, starts=None, act=True):
    """One batch row: x [T, D], weight [D, K], state [K-1, D]; (y, last K-1 rows)."""
    T, D = x.shape
    K = weight.shape[1]
    rows = np.concatenate([np.zeros((K - 1, D)) if state is None else state, x])
    doc = _documents(np.zeros(T) if starts is None else starts, K)
    s = np.zeros((T, D)) + (0.0 if bias is None else bias)
    for t in range(T):
        for k in range(K):
            if doc[t + k] == doc[t + K - 1]:
                s[t] = s[t] + weight[:, k] * rows[t + k]
    last = np.where((doc[T:] == doc[-1])[:, None], rows[T:], 0.0)
    return (silu(s) if act else s), last


def short_conv_gradients(dy, x, weight, bias=None, state=None, dlast=None, starts=None, act=True):
    T, D = x.shape
    K = weight.shape[1]
    rows = np.concatenate([np.zeros((K - 1, D)) if state is None else state, x])
    doc = _documents(np.zeros(T) if starts is None else starts, K)
    s, _ = short_conv(x, weight, bias, state, starts, act=False)
    ds = dy * (silu_slope(s) if act else 1.0)
    drows, dw = np.zeros_like(rows), np.zeros_like(weight)
    for t in range(T):
        for k in range(K):
            if doc[t + k] == doc[t + K - 1]:
                drows[t + k] += weight[:, k] * ds[t]
                dw[:, k] += ds[t] * rows[t + k]
    if dlast is not None:
        drows[T:] += np.where((doc[T:] == doc[-1])[:, None], dlast, 0.0)
    return {"x": drows[K - 1:], "state": drows[:K - 1], "weight": dw, "bias": ds.sum(0)}


# ------------------------------------------------------------------ state space recurrence

def state_space(x, dt, A, B, C, h0=None, skip=None, z=None, dt_bias=None, plus=True, starts=None):
    """One batch row: x, dt, z [T, D], A [D, N], B, C [T, G, N]. Returns y [T, D] and the
    states [T + 1, D, N] (entry 0 is the start)."""
    T, D = x.shape
    N, per = A.shape[1], D // B.shape[1]
    u = dt + (0.0 if dt_bias is None else dt_bias)
    if plus:
        u = softplus(u)
    h = np.zeros((T + 1, D, N))
    if h0 is not None:
        h[0] = h0
    y = np.zeros((T, D))
    for t in range(T):
        b, c = np.repeat(B[t], per, 0), np.repeat(C[t], per, 0)
        old = np.zeros_like(h[t]) if starts is not None and starts[t] else h[t]
        h[t + 1] = np.exp(u[t][:, None] * A) * old + (u[t] * x[t])[:, None] * b
        y[t] = (c * h[t + 1]).sum(1) + (0.0 if skip is None else skip * x[t])
    return (y if z is None else y * silu(z)), h


def state_space_gradients(dy, x, dt, A, B, C, h0=None, dhT=None, skip=None, z=None, dt_bias=None,
                          plus=True, starts=None):
    T, D = x.shape
    G = B.shape[1]
    per = D // G
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    u = softplus(raw) if plus else raw
    y, h = state_space(x, dt, A, B, C, h0, skip, None, dt_bias, plus, starts)
    out = {n: np.zeros_like(v) for n, v in (("x", x), ("dt", dt), ("A", A), ("B", B), ("C", C))}
    p = dy if z is None else dy * silu(z)
    if z is not None:
        out["z"] = dy * y * silu_slope(z)
    E = np.zeros_like(A) if dhT is None else np.array(dhT)
    for t in range(T - 1, -1, -1):
        b, c = np.repeat(B[t], per, 0), np.repeat(C[t], per, 0)
        a = np.exp(u[t][:, None] * A)
        if starts is not None and starts[t]:
            a = np.zeros_like(a)
        E = E + c * p[t][:, None]                      # the gradient of h_t
        out["C"][t] = (h[t + 1] * p[t][:, None]).reshape(G, per, -1).sum(1)
        out["B"][t] = (E * (u[t] * x[t])[:, None]).reshape(G, per, -1).sum(1)
        da = E * a * h[t]                              # times d(u A)
        out["A"] += da * u[t][:, None]
        eb = (E * b).sum(1)
        du = (da * A).sum(1) + x[t] * eb
        out["x"][t] = u[t] * eb + (0.0 if skip is None else skip * p[t])
        out["dt"][t] = du * (sigmoid(raw[t]) if plus else 1.0)
        E = a * E
    out["h0"] = E
    out["skip"] = (p * x).sum(0)
    out["dt_bias"] = out["dt"].sum(0)
    return out


# ------------------------------------------------------------------ norms around a block

def _rms(x, eps):
    return np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def block_sum(x, residual, post, gate=None, scale=None, eps=1e-6):
    u = x / _rms(x, eps) * post
    if scale is not None:
        u = u * scale
    if gate is not None:
        u = u * sigmoid(gate)
    return residual + u


def pre_norm(r, pre, eps=1e-6):
    return r / _rms(r, eps) * pre


def _norm_back(dy, x, w, eps):
    rms = _rms(x, eps)
    n, dn = x / rms, dy * w
    return (dn - n * np.mean(dn * n, axis=-1, keepdims=True)) / rms


def block_norms_gradients(dy, x, r, post, pre, gate=None, scale=None, dres=None, eps=1e-6):
    dr = _norm_back(dy, r, pre, eps) + (0.0 if dres is None else dres)
    n = x / _rms(x, eps)
    s = 1.0 if scale is None else scale
    g = np.ones_like(x) if gate is None else sigmoid(gate)
    return {"residual": dr, "pre": (dy * r / _rms(r, eps)).sum(0), "post": (dr * s * g * n).sum(0),
            "scale": (dr * g * n * post).sum(0), "gate": dr * s * n * post * g * (1.0 - g),
            "x": _norm_back(dr * s * g, x, post, eps)}
