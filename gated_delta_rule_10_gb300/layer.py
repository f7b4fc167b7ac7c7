"""The layer operators around the delta rule: linear attention with a decay for
each head, the residual RMS norm and the rotary positions.

Argument marshalling only, as in ``_binding``: every step runs in the library's
CUDA kernels behind ``include/gdr.h``, and there is no fallback.
"""
import ctypes

import torch

from ._binding import GDR_BF16, GDR_F32, GdrError, _check as _check_slow, _vp, lib

_ll, _sz, _int, _f32 = ctypes.c_longlong, ctypes.c_size_t, ctypes.c_int, ctypes.c_float


class DecayShape(ctypes.Structure):
    """Mirror of ``gdr_decay_shape``."""
    _fields_ = [(n, _int) for n in ("B", "T", "H", "Hk", "dk", "dv", "dtype",
                                    "decay_per_head")] + \
               [("scale", _f32)] + [(n, _ll) for n in ("q_stride", "k_stride", "v_stride")]


class RotaryShape(ctypes.Structure):
    """Mirror of ``gdr_rotary_shape``."""
    _fields_ = [(n, _int) for n in ("B", "T", "H", "Hk", "d", "rot", "dtype", "interleaved",
                                    "inverse", "start", "table_length")] + \
               [(n, _ll) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")]


class RotaryScaling(ctypes.Structure):
    """Mirror of ``gdr_rotary_scaling``."""
    _fields_ = [("kind", _int), ("factor", ctypes.c_double), ("original_length", _int),
                ("fast", ctypes.c_double), ("slow", ctypes.c_double),
                ("magnitude", ctypes.c_double)]


_KINDS = {None: 0, "linear": 1, "base": 2, "ramp": 3}
_fns = None


def _lib():
    """The library with these entries' argument types set."""
    global _fns
    if _fns is None:
        L = lib()
        dp, rp, zp = (ctypes.POINTER(t) for t in (DecayShape, RotaryShape, _sz))
        for name, args in (
                ("gdr_decay_chunk_fwd_workspace", [dp, zp]),
                ("gdr_decay_chunk_fwd", [dp] + [_vp] * 8 + [_sz, _vp]),
                ("gdr_decay_chunk_bwd_workspace", [dp, zp]),
                ("gdr_decay_chunk_bwd", [dp] + [_vp] * 13 + [_sz, _vp]),
                ("gdr_decay_step", [dp] + [_vp] * 7),
                ("gdr_add_rmsnorm", [_ll, _int, _int, _vp, _vp, _vp, _f32, _vp, _vp, _vp]),
                ("gdr_add_rmsnorm_fp8", [_ll, _int, _int, _vp, _vp, _vp, _f32, _vp, _vp, _vp,
                                         _vp]),
                ("gdr_add_rmsnorm_bwd_workspace", [_ll, _int, zp]),
                ("gdr_add_rmsnorm_bwd", [_ll, _int, _int, _vp, _vp, _vp, _f32, _vp, _vp, _vp,
                                         _vp, _sz, _vp]),
                ("gdr_rotary", [rp] + [_vp] * 8),
                ("gdr_rotary_table", [_int, _int, ctypes.c_double,
                                      ctypes.POINTER(RotaryScaling), _vp, _vp, _vp])):
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = _int
        _fns = L
    return _fns


# A decode step makes these calls once per layer: the common case of each helper
# below is a few attribute reads.

def _call(name, device, *args):
    fn = getattr(_fns or _lib(), name)
    if device.index == torch.cuda.current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st:
        raise GdrError(st, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(t, name, dtype, device, shape=None):
    if t is None or (t.dtype is dtype and t.device == device and device.type == "cuda" and
                     t.is_contiguous() and (shape is None or t.shape == shape)):
        return
    _check_slow(t, name, dtype, device, shape)


def _dtype(t):
    if t.dtype is torch.bfloat16:
        return GDR_BF16
    if t.dtype is torch.float32:
        return GDR_F32
    raise ValueError("expected bf16 or fp32, got %s" % t.dtype)


def _used_on(stream, device, *tensors):
    """Tensors made here are used on `stream`: where that is not the stream they
    were made on, their memory is kept until its work is done."""
    if stream is None:
        return
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream != torch.cuda.current_stream(device):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _rows(t, name, dtype, device, shape):
    """Checks a [B, T, heads, d] tensor whose heads and channels are dense and
    whose tokens are evenly spaced over the batch; returns elements per token."""
    if t.dtype is dtype and t.device == device and t.is_cuda and t.shape == shape and \
            t.is_contiguous():
        return 0
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be a CUDA tensor on %s" % (name, device))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    B, T, H, d = shape
    sb, st, sh, sd = t.stride()
    step = st if T > 1 else sb
    if (d > 1 and sd != 1) or (H > 1 and sh != d) or (T > 1 and B > 1 and sb != T * st) or \
            step < H * d:
        raise ValueError("%s must have dense heads and evenly spaced tokens" % name)
    return step


def _tokens(t, name, dtype, device, shape):
    """_rows of an [N, heads, d] tensor: one token of each of N sequences."""
    if t.dtype is dtype and t.device == device and t.is_cuda and t.shape == shape and \
            t.is_contiguous():
        return 0
    if t.dim() != 3:
        raise ValueError("%s must be [N, heads, d]" % name)
    return _rows(t.unsqueeze(1), name, dtype, device, (shape[0], 1) + tuple(shape[1:]))


def _new_or(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device), True
    _check(t, name, dtype, device, shape)
    return t, False


def _workspace_bytes(t, device):
    """Bytes of a caller's workspace (None: 0), which the kernels write as it stands."""
    if t is None:
        return 0
    if not t.is_cuda or t.device != device:
        raise ValueError("workspace must be a CUDA tensor on %s" % (device,))
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.numel() * t.element_size()


def _decay_shape(q, k, v, g, scale):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [B, T, heads, d]")
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    dev, dt = q.device, q.dtype
    s = DecayShape(B, T, H, Hk, dk, dv, _dtype(q), int(g.dim() == 1),
                   float(dk ** -0.5 if scale is None else scale),
                   _rows(q, "q", dt, dev, (B, T, Hk, dk)), _rows(k, "k", dt, dev, (B, T, Hk, dk)),
                   _rows(v, "v", dt, dev, (B, T, H, dv)))
    _check(g, "g", torch.float32, dev, (H,) if g.dim() == 1 else (B, T, H))
    return s


def decay_chunk_fwd_workspace_bytes(shape):
    n = _sz(0)
    st = (_fns or _lib()).gdr_decay_chunk_fwd_workspace(ctypes.byref(shape), ctypes.byref(n))
    if st:
        raise GdrError(st, "gdr_decay_chunk_fwd_workspace")
    return n.value


def decay_chunk_bwd_workspace_bytes(shape):
    n = _sz(0)
    st = _lib().gdr_decay_chunk_bwd_workspace(ctypes.byref(shape), ctypes.byref(n))
    if st:
        raise GdrError(st, "gdr_decay_chunk_bwd_workspace")
    return n.value


def decay_chunk_fwd(q, k, v, g, h0=None, *, scale=None, output_final_state=True, o=None, hT=None,
                    workspace=None, stream=None):
    """Linear attention with a decay for each head over whole prompts
    (``gdr_decay_chunk_fwd``): S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k: [B, T, Hk, d_k]; v: [B, T, H, d_v] (bf16 or fp32, one dtype), H a multiple
    of Hk; parts of a fused projection (dense heads, evenly spaced tokens) are taken
    as they are. g: [B, T, H] or [H] fp32 log-decay, -inf clears the state; h0:
    [B, H, d_k, d_v] fp32 or None. ``scale`` defaults to d_k^-1/2. Returns (o, hT),
    hT None unless requested.
    """
    s = _decay_shape(q, k, v, g, scale)
    dev, dt = q.device, q.dtype
    _check(h0, "h0", torch.float32, dev, (s.B, s.H, s.dk, s.dv))
    o, new_o = _new_or(o, "o", (s.B, s.T, s.H, s.dv), dt, dev)
    new_h = False
    if hT is not None or output_final_state:
        hT, new_h = _new_or(hT, "hT", (s.B, s.H, s.dk, s.dv), torch.float32, dev)
    ws = None
    need = decay_chunk_fwd_workspace_bytes(s)
    if workspace is None and need:
        ws = workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _call("gdr_decay_chunk_fwd", dev, ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
          _ptr(h0), _ptr(o), _ptr(hT), _ptr(workspace), _workspace_bytes(workspace, dev),
          _stream(stream, dev))
    _used_on(stream, dev, ws, o if new_o else None, hT if new_h else None)
    return o, hT


def decay_chunk_bwd(q, k, v, g, dO, h0=None, dhT=None, *, scale=None, workspace=None,
                    stream=None):
    """Gradients of ``decay_chunk_fwd`` (``gdr_decay_chunk_bwd``) for the loss
    <dO, o> + <dhT, hT>: a dict with q, k, v (the inputs' dtype), g (fp32, g's
    shape) and h0 (fp32)."""
    s = _decay_shape(q, k, v, g, scale)
    dev, dt = q.device, q.dtype
    _check(dO, "dO", dt, dev, (s.B, s.T, s.H, s.dv))
    _check(h0, "h0", torch.float32, dev, (s.B, s.H, s.dk, s.dv))
    _check(dhT, "dhT", torch.float32, dev, (s.B, s.H, s.dk, s.dv))
    out = {"q": torch.empty(s.B, s.T, s.Hk, s.dk, dtype=dt, device=dev),
           "k": torch.empty(s.B, s.T, s.Hk, s.dk, dtype=dt, device=dev),
           "v": torch.empty(s.B, s.T, s.H, s.dv, dtype=dt, device=dev),
           "g": torch.empty(g.shape, dtype=torch.float32, device=dev),
           "h0": torch.empty(s.B, s.H, s.dk, s.dv, dtype=torch.float32, device=dev)}
    ws = None
    if workspace is None:
        ws = workspace = torch.empty(decay_chunk_bwd_workspace_bytes(s), dtype=torch.uint8,
                                     device=dev)
    _call("gdr_decay_chunk_bwd", dev, ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
          _ptr(h0), _ptr(dO), _ptr(dhT), *(_ptr(out[n]) for n in ("q", "k", "v", "g", "h0")),
          _ptr(workspace), _workspace_bytes(workspace, dev), _stream(stream, dev))
    _used_on(stream, dev, ws, *out.values())
    return out


def decay_step(q, k, v, g, state, *, scale=None, o=None, stream=None):
    """One decode step (``gdr_decay_step``); updates ``state`` in place.

    q, k: [N, Hk, d_k]; v: [N, H, d_v]; g: [N, H] or [H] fp32; state:
    [N, H, d_k, d_v] fp32. Returns o [N, H, d_v].
    """
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [N, heads, d]")
    N, H, dv = v.shape
    Hk, dk = q.shape[1], q.shape[2]
    dev, dt = q.device, q.dtype
    s = DecayShape(N, 1, H, Hk, dk, dv, _dtype(q), int(g.dim() == 1),
                   float(dk ** -0.5 if scale is None else scale), _tokens(q, "q", dt, dev, (N, Hk, dk)),
                   _tokens(k, "k", dt, dev, (N, Hk, dk)), _tokens(v, "v", dt, dev, (N, H, dv)))
    _check(g, "g", torch.float32, dev, (H,) if g.dim() == 1 else (N, H))
    _check(state, "state", torch.float32, dev, (N, H, dk, dv))
    o, new_o = _new_or(o, "o", (N, H, s.dv), q.dtype, dev)
    _call("gdr_decay_step", dev, ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state),
          _ptr(o), _stream(stream, dev))
    _used_on(stream, dev, o if new_o else None)
    return o


def _norm_inputs(x, residual, weight):
    D = x.shape[-1]
    _check(x, "x", x.dtype, x.device)
    _check(residual, "residual", x.dtype, x.device, tuple(x.shape))
    _check(weight, "weight", torch.float32, x.device, (D,))
    return x.numel() // D if D else 0, D, _dtype(x)


def add_rmsnorm(x, residual, weight, eps=1e-6, *, out=None, residual_out=None, stream=None):
    """Residual addition and RMS norm over the last axis (``gdr_add_rmsnorm``):
    r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight. x, residual:
    [..., D] bf16 or fp32; weight: [D] fp32. Returns (y, r); ``residual_out`` may be
    x or residual itself (in place)."""
    rows, D, dt = _norm_inputs(x, residual, weight)
    y, new_y = _new_or(out, "out", tuple(x.shape), x.dtype, x.device)
    r, new_r = _new_or(residual_out, "residual_out", tuple(x.shape), x.dtype, x.device)
    if rows and y.data_ptr() == r.data_ptr():
        raise ValueError("out and residual_out must be apart")
    _call("gdr_add_rmsnorm", x.device, rows, D, dt, _ptr(x), _ptr(residual), _ptr(weight),
          float(eps), _ptr(r), _ptr(y), _stream(stream, x.device))
    _used_on(stream, x.device, y if new_y else None, r if new_r else None)
    return y, r


def add_rmsnorm_fp8(x, residual, weight, eps=1e-6, *, residual_out=None, stream=None):
    """``add_rmsnorm`` with y in 8 bits (``gdr_add_rmsnorm_fp8``): returns (y8, scales,
    r), y8 [..., D] float8_e4m3fn and scales [..., ceil(D / 128)] fp32 with
    y = y8 * scales of its 128-column block."""
    rows, D, dt = _norm_inputs(x, residual, weight)
    dev = x.device
    y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.empty(x.shape[:-1] + (-(-D // 128),), dtype=torch.float32, device=dev)
    r, new_r = _new_or(residual_out, "residual_out", tuple(x.shape), x.dtype, dev)
    _call("gdr_add_rmsnorm_fp8", dev, rows, D, dt, _ptr(x), _ptr(residual), _ptr(weight),
          float(eps), _ptr(r), _ptr(y), _ptr(scales), _stream(stream, dev))
    _used_on(stream, dev, y, scales, r if new_r else None)
    return y, scales, r


def add_rmsnorm_bwd(dy, sum, weight, eps=1e-6, *, dres=None, dx=None, workspace=None,
                    stream=None):
    """Gradients of ``add_rmsnorm`` (``gdr_add_rmsnorm_bwd``): dy of y and, if given,
    dres of r = ``sum``. Returns (dx, dweight): dx is the gradient of x and of the
    residual alike, dweight [D] fp32."""
    rows, D, dt = _norm_inputs(dy, sum, weight)
    dev = dy.device
    _check(dres, "dres", dy.dtype, dev, tuple(dy.shape))
    dx, new_x = _new_or(dx, "dx", tuple(dy.shape), dy.dtype, dev)
    dw = torch.empty(D, dtype=torch.float32, device=dev)
    ws = None
    if workspace is None:
        n = _sz(0)
        st = _lib().gdr_add_rmsnorm_bwd_workspace(rows, D, ctypes.byref(n))
        if st:
            raise GdrError(st, "gdr_add_rmsnorm_bwd_workspace")
        ws = workspace = torch.empty(n.value, dtype=torch.uint8, device=dev)
    _call("gdr_add_rmsnorm_bwd", dev, rows, D, dt, _ptr(dy), _ptr(sum), _ptr(weight), float(eps),
          _ptr(dres), _ptr(dx), _ptr(dw), _ptr(workspace), _workspace_bytes(workspace, dev),
          _stream(stream, dev))
    _used_on(stream, dev, ws, dw, dx if new_x else None)
    return dx, dw


def rotary_table(length, rot, base=10000.0, *, scaling=None, factor=1.0, original_length=0,
                 fast=32.0, slow=1.0, magnitude=None, device="cuda", stream=None):
    """cos and sin tables [length, rot / 2] fp32 for ``rotary`` (``gdr_rotary_table``).

    ``scaling`` for contexts longer than trained: None, "linear" (positions divided
    by factor), "base" (the base raised) or "ramp" (frequencies that turn ``fast``
    times over ``original_length`` kept, those that turn ``slow`` times divided by
    factor, a ramp between; cos and sin times ``magnitude``, by default
    0.1 ln(factor) + 1; both after "YaRN", Peng et al.).
    """
    if scaling not in _KINDS:
        raise ValueError("unknown scaling %r" % (scaling,))
    if magnitude is None:
        magnitude = 0.1 * float(torch.log(torch.tensor(float(factor), dtype=torch.float64))) + 1.0
    dev = torch.device(device)
    cos = torch.empty(length, rot // 2, dtype=torch.float32, device=dev)
    sin = torch.empty_like(cos)
    z = RotaryScaling(_KINDS[scaling], float(factor), int(original_length), float(fast),
                      float(slow), float(magnitude))
    _call("gdr_rotary_table", cos.device, int(length), int(rot), float(base), ctypes.byref(z),
          _ptr(cos), _ptr(sin), _stream(stream, cos.device))
    _used_on(stream, cos.device, cos, sin)
    return cos, sin


def rotary(q, k, cos, sin, positions=None, *, start=0, interleaved=False, inverse=False,
           q_out=None, k_out=None, stream=None):
    """Rotary positions of q [B, T, H, d] and k [B, T, Hk, d] (``gdr_rotary``): the
    first 2 * cos.shape[1] channels of every head turn by their token's angles.

    cos, sin: [length, rot / 2] fp32 (``rotary_table``); positions: [B, T] int32 or
    None for start + t. ``interleaved`` pairs neighbouring channels, else channels j
    and j + rot/2. ``inverse`` turns back (the gradient). Parts of a fused projection
    are taken as they are; q_out and k_out may be q and k (in place). Returns (q, k).
    """
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, T, heads, d]")
    B, T, H, d = q.shape
    Hk = k.shape[2]
    dev, dt = q.device, q.dtype
    sq = _rows(q, "q", dt, dev, (B, T, H, d))
    sk = _rows(k, "k", dt, dev, (B, T, Hk, d))
    if cos.dim() != 2:
        raise ValueError("cos and sin must be [length, rot / 2]")
    _check(cos, "cos", torch.float32, dev)
    _check(sin, "sin", torch.float32, dev, tuple(cos.shape))
    _check(positions, "positions", torch.int32, dev, (B, T))
    new = []
    outs = []
    for t, given, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
        if given is None:
            given = torch.empty(t.shape, dtype=dt, device=dev)
            new.append(given)
        outs.append((given, _rows(given, name, dt, dev, tuple(t.shape))))
    (qo, sqo), (ko, sko) = outs
    s = RotaryShape(B, T, H, Hk, d, 2 * cos.shape[1], _dtype(q), int(interleaved), int(inverse),
                    int(start), cos.shape[0], sq, sk, sqo, sko)
    _call("gdr_rotary", dev, ctypes.byref(s), _ptr(q), _ptr(k), _ptr(cos), _ptr(sin),
          _ptr(positions), _ptr(qo), _ptr(ko), _stream(stream, dev))
    _used_on(stream, dev, *new)
    return qo, ko
