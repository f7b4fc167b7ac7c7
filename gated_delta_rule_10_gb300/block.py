"""The operators of a block around a recurrence: the short causal convolution, the state
space recurrence and the norms after and before the block.

Argument marshalling only, as in ``layer``: every step runs in the library's CUDA kernels
behind ``include/gdr.h``, and there is no fallback.
"""
import ctypes

import torch

from ._binding import GDR_BF16, GDR_F32, GdrError, _check as _check_slow, _vp, lib
from .layer import _f32, _int, _ll, _ptr, _sz, _used_on, _workspace_bytes

F32, BF16 = torch.float32, torch.bfloat16


class ConvShape(ctypes.Structure):
    """Mirror of ``gdr_conv_shape``."""
    _fields_ = [(n, _int) for n in ("B", "T", "D", "K", "dtype", "silu")] + [("x_stride", _ll)]


class StateSpaceShape(ctypes.Structure):
    """Mirror of ``gdr_state_space_shape``."""
    _fields_ = [(n, _int) for n in ("B", "T", "D", "G", "N", "dtype", "softplus")] + \
               [(n, _ll) for n in ("x_stride", "dt_stride", "z_stride", "b_stride", "c_stride")]


_fns = None


def _lib():
    """The library with these entries' argument types set."""
    global _fns
    if _fns is None:
        L = lib()
        cp, sp, zp = (ctypes.POINTER(t) for t in (ConvShape, StateSpaceShape, _sz))
        for name, args in (
                ("gdr_short_conv_fwd", [cp] + [_vp] * 8),
                ("gdr_short_conv_bwd_workspace", [cp, zp]),
                ("gdr_short_conv_bwd", [cp] + [_vp] * 12 + [_sz, _vp]),
                ("gdr_short_conv_step", [cp] + [_vp] * 6),
                ("gdr_state_space_fwd_workspace", [sp, zp]),
                ("gdr_state_space_fwd", [sp] + [_vp] * 13 + [_sz, _vp]),
                ("gdr_state_space_bwd_workspace", [sp, zp]),
                ("gdr_state_space_bwd", [sp] + [_vp] * 22 + [_sz, _vp]),
                ("gdr_state_space_step", [sp] + [_vp] * 11),
                ("gdr_block_norms", [_ll, _int, _int] + [_vp] * 6 + [_f32] + [_vp] * 3),
                ("gdr_block_norms_bwd_workspace", [_ll, _int, zp]),
                ("gdr_block_norms_bwd", [_ll, _int, _int] + [_vp] * 8 + [_f32] + [_vp] * 7 +
                 [_sz, _vp])):
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = _int
        _fns = L
    return _fns


def _bytes(name, *args):
    """A workspace query."""
    n = _sz(0)
    st = getattr(_fns or _lib(), name)(*args, ctypes.byref(n))
    if st:
        raise GdrError(st, name)
    return n.value


# A decode step makes these calls once per layer: as in ``layer``, the common case of each
# helper is a few attribute reads.

def _run(name, device, *args):
    fn = getattr(_fns or _lib(), name)
    if device.index == torch.cuda.current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st:
        raise GdrError(st, name)


def _dtype(t):
    """The library's number of the type of `t`, an operator's main input on the GPU."""
    dt = t.dtype
    if dt is not BF16 and dt is not F32:
        raise ValueError("expected bf16 or fp32, got %s" % dt)
    if not t.is_cuda:
        raise ValueError("x must be a CUDA tensor, got one on %s" % t.device)
    return GDR_BF16 if dt is BF16 else GDR_F32


def _check(t, name, dtype, device, shape):
    """A contiguous tensor like this on `device` (a GPU), or None."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and
                     t.is_contiguous()):
        return
    _check_slow(t, name, dtype, device, shape)


def _new_or(t, name, like, dtype=None, shape=None):
    """`t` as the caller gave it, or a new tensor like `like`; and whether it is new."""
    if t is None:
        if shape is None:
            return torch.empty_like(like, memory_format=torch.contiguous_format), True
        return torch.empty(shape, dtype=dtype, device=like.device), True
    if shape is None:
        return _given(t, name, like), False
    _check(t, name, dtype, like.device, shape)
    return t, False


def _given(t, name, like):
    """A caller's output, to be as `like`."""
    _check(t, name, like.dtype, like.device, like.shape)
    return t


def _stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _rows(t, name, dtype, device, shape):
    """Checks a tensor [B, T, ...] ([N, ...] for single tokens) whose tokens are dense
    inside and evenly spaced; returns elements per token (0: dense)."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return 0
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be a CUDA tensor on %s" % (name, device))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return None


def _tokens(t, name, dtype, device, shape, lead=2):
    """_rows with `lead` leading token axes (2: batch rows and tokens; 1: sequences)."""
    step = _rows(t, name, dtype, device, shape)
    if step is not None:
        return step
    stride = t.stride()
    inner = 1
    for n, s in zip(reversed(shape[lead:]), reversed(stride[lead:])):
        if n > 1 and s != inner:
            raise ValueError("%s must have dense, evenly spaced tokens" % name)
        inner *= n
    B, T = (shape[0], shape[1]) if lead == 2 else (1, shape[0])
    sb, st = (stride[0], stride[1]) if lead == 2 else (0, stride[0])
    step = st if T > 1 else (sb if B > 1 else inner)
    if (T > 1 and B > 1 and sb != T * st) or step < inner:
        raise ValueError("%s must have dense, evenly spaced tokens" % name)
    return step


def _starts(t, device, shape):
    """The documents' starts: bool or uint8, nonzero at a document's first token."""
    if t is None:
        return
    if t.dtype not in (torch.bool, torch.uint8):
        raise ValueError("starts must be bool or uint8, got %s" % t.dtype)
    _check(t, "starts", t.dtype, device, shape)


# ------------------------------------------------------------------ short convolution

def _conv_shape(x, weight, bias, silu, lead):
    if x.dim() != lead + 1 or weight.dim() != 2:
        raise ValueError("x must be [%s, D] and weight [D, K]" % ("B, T" if lead == 2 else "N"))
    shape = x.shape
    D, K = weight.shape
    if shape[-1] != D:
        raise ValueError("weight has %d channels, x %d" % (D, shape[-1]))
    dev, dt = x.device, _dtype(x)
    _check(weight, "weight", F32, dev, (D, K))
    _check(bias, "bias", F32, dev, (D,))
    return ConvShape(shape[0], shape[1] if lead == 2 else 1, D, K, dt, int(bool(silu)),
                     _tokens(x, "x", x.dtype, dev, shape, lead))


def short_conv_bwd_workspace_bytes(shape):
    return _bytes("gdr_short_conv_bwd_workspace", ctypes.byref(shape))


def short_conv_fwd(x, weight, bias=None, state=None, *, starts=None, silu=True,
                   output_final_state=True, y=None, state_out=None, stream=None):
    """Short causal convolution over the tokens (``gdr_short_conv_fwd``): s_t = bias +
    sum_j weight[:, K-1-j] x_{t-j}, y = silu(s), or s without ``silu``.

    x: [B, T, D] (bf16 or fp32; a part of a projection is taken as it is); weight: [D, K]
    fp32, K from 2 to 4; bias: [D] fp32 or None; state: [B, K-1, D] in x's dtype, the rows
    before the first token, or None for zeros; starts: [B, T] bool or uint8, nonzero at a
    document's first token, whose taps do not reach behind it. Returns (y, state_out): the
    last K - 1 rows (zeros where they are of an earlier document), None unless requested.
    """
    s = _conv_shape(x, weight, bias, silu, 2)
    dev, dt = x.device, x.dtype
    edge = (s.B, s.K - 1, s.D)
    _check(state, "state", dt, dev, edge)
    _starts(starts, dev, (s.B, s.T))
    y, new_y = _new_or(y, "y", x)
    new_s = False
    if state_out is not None or output_final_state:
        state_out, new_s = _new_or(state_out, "state_out", x, dt, edge)
    _run("gdr_short_conv_fwd", dev, ctypes.byref(s), _ptr(x), _ptr(weight), _ptr(bias),
         _ptr(starts), _ptr(state), _ptr(y), _ptr(state_out), _stream(stream, dev))
    _used_on(stream, dev, y if new_y else None, state_out if new_s else None)
    return y, state_out


def short_conv_bwd(dy, x, weight, bias=None, state=None, dstate=None, *, starts=None, silu=True,
                   workspace=None, stream=None):
    """Gradients of ``short_conv_fwd`` (``gdr_short_conv_bwd``) for the loss <dy, y> +
    <dstate, state_out>: a dict with x and state (x's dtype), weight and bias (fp32)."""
    s = _conv_shape(x, weight, bias, silu, 2)
    dev, dt = x.device, x.dtype
    edge = (s.B, s.K - 1, s.D)
    _check(state, "state", dt, dev, edge)
    _check(dstate, "dstate", dt, dev, edge)
    _check(dy, "dy", dt, dev, x.shape)
    _starts(starts, dev, (s.B, s.T))
    out = {"x": torch.empty(x.shape, dtype=dt, device=dev),
           "weight": torch.empty(weight.shape, dtype=F32, device=dev),
           "bias": torch.empty(s.D, dtype=F32, device=dev),
           "state": torch.empty(edge, dtype=dt, device=dev)}
    ws = None
    if workspace is None:
        ws = workspace = torch.empty(short_conv_bwd_workspace_bytes(s), dtype=torch.uint8,
                                     device=dev)
    _run("gdr_short_conv_bwd", dev, ctypes.byref(s), _ptr(x), _ptr(weight), _ptr(bias),
         _ptr(starts), _ptr(state), _ptr(dy), _ptr(dstate),
         *(_ptr(out[n]) for n in ("x", "weight", "bias", "state")), _ptr(workspace),
         _workspace_bytes(workspace, dev), _stream(stream, dev))
    _used_on(stream, dev, ws, *out.values())
    return out


def short_conv_step(x, weight, bias, state, *, silu=True, y=None, stream=None):
    """One token of each sequence (``gdr_short_conv_step``): x [N, D], state [N, K-1, D],
    moved on by one row in place. Returns y [N, D]."""
    s = _conv_shape(x, weight, bias, silu, 1)
    dev = x.device
    if state is None:
        raise ValueError("state is needed")
    _check(state, "state", x.dtype, dev, (s.B, s.K - 1, s.D))
    out = torch.empty_like(x, memory_format=torch.contiguous_format) if y is None else \
        _given(y, "y", x)
    _run("gdr_short_conv_step", dev, ctypes.byref(s), x.data_ptr(), weight.data_ptr(), _ptr(bias),
         state.data_ptr(), out.data_ptr(), _stream(stream, dev))
    if y is None and stream is not None:
        _used_on(stream, dev, out)
    return out


# ------------------------------------------------------------------ state space recurrence

def _space_shape(x, dt, A, B, C, skip, z, dt_bias, softplus, lead):
    if x.dim() != lead + 1 or A.dim() != 2 or B.dim() != lead + 2:
        raise ValueError("x must be [%s, D], A [D, N], B and C [%s, G, N]"
                         % (("B, T",) * 2 if lead == 2 else ("N",) * 2))
    shape = tuple(x.shape)
    D, N = A.shape
    dev, t = x.device, x.dtype
    if shape[-1] != D:
        raise ValueError("A has %d channels, x %d" % (D, shape[-1]))
    bc = shape[:lead] + (B.shape[lead], N)
    s = StateSpaceShape(shape[0], shape[1] if lead == 2 else 1, D, bc[lead], N, _dtype(x),
                        int(bool(softplus)), _tokens(x, "x", t, dev, shape, lead),
                        _tokens(dt, "dt", t, dev, shape, lead),
                        0 if z is None else _tokens(z, "z", t, dev, shape, lead),
                        _tokens(B, "B", t, dev, bc, lead), _tokens(C, "C", t, dev, bc, lead))
    _check(A, "A", F32, dev, (D, N))
    _check(skip, "skip", F32, dev, (D,))
    _check(dt_bias, "dt_bias", F32, dev, (D,))
    return s


def state_space_fwd_workspace_bytes(shape):
    return _bytes("gdr_state_space_fwd_workspace", ctypes.byref(shape))


def state_space_bwd_workspace_bytes(shape):
    return _bytes("gdr_state_space_bwd_workspace", ctypes.byref(shape))


def state_space_fwd(x, dt, A, B, C, h0=None, *, skip=None, z=None, dt_bias=None, softplus=True,
                    starts=None, output_final_state=True, y=None, hT=None, workspace=None,
                    stream=None):
    """State space recurrence with a decay for each token, channel and state
    (``gdr_state_space_fwd``): u = softplus(dt + dt_bias), h_t = exp(u A) h_{t-1} + u x B_t,
    y = (C_t h_t + skip x) silu(z).

    x, dt, z: [B, T, D]; B, C: [B, T, G, N] (bf16 or fp32, one dtype; parts of projections
    are taken as they are), a group's D / G channels share theirs; A: [D, N], skip, dt_bias:
    [D] fp32; h0: [B, D, N] fp32 or None. Without ``softplus`` u = dt + dt_bias. starts:
    [B, T] bool or uint8, nonzero at a document's first token, which clears the state.
    Returns (y, hT), hT None unless requested.
    """
    s = _space_shape(x, dt, A, B, C, skip, z, dt_bias, softplus, 2)
    dev = x.device
    _check(h0, "h0", F32, dev, (s.B, s.D, s.N))
    _starts(starts, dev, (s.B, s.T))
    y, new_y = _new_or(y, "y", x)
    new_h = False
    if hT is not None or output_final_state:
        hT, new_h = _new_or(hT, "hT", x, F32, (s.B, s.D, s.N))
    ws = None
    need = state_space_fwd_workspace_bytes(s)
    if workspace is None and need:
        ws = workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _run("gdr_state_space_fwd", dev, ctypes.byref(s), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
         _ptr(skip), _ptr(z), _ptr(dt_bias), _ptr(starts), _ptr(h0), _ptr(y), _ptr(hT),
         _ptr(workspace), _workspace_bytes(workspace, dev), _stream(stream, dev))
    _used_on(stream, dev, ws, y if new_y else None, hT if new_h else None)
    return y, hT


def state_space_bwd(dy, x, dt, A, B, C, h0=None, dhT=None, *, skip=None, z=None, dt_bias=None,
                    softplus=True, starts=None, workspace=None, stream=None):
    """Gradients of ``state_space_fwd`` (``gdr_state_space_bwd``) for the loss <dy, y> +
    <dhT, hT>: a dict with x, dt, B, C, z (their dtype) and A, skip, dt_bias, h0 (fp32);
    skip, z and dt_bias are None where they were not given."""
    s = _space_shape(x, dt, A, B, C, skip, z, dt_bias, softplus, 2)
    dev, t = x.device, x.dtype
    _check(h0, "h0", F32, dev, (s.B, s.D, s.N))
    _check(dhT, "dhT", F32, dev, (s.B, s.D, s.N))
    _check(dy, "dy", t, dev, x.shape)
    _starts(starts, dev, (s.B, s.T))
    new = lambda like, d: None if like is None else torch.empty(like.shape, dtype=d, device=dev)  # noqa: E731
    out = {"x": new(x, t), "dt": new(dt, t), "A": new(A, F32), "B": new(B, t), "C": new(C, t),
           "skip": new(skip, F32), "z": new(z, t), "dt_bias": new(dt_bias, F32),
           "h0": torch.empty(s.B, s.D, s.N, dtype=F32, device=dev)}
    ws = None
    if workspace is None:
        ws = workspace = torch.empty(state_space_bwd_workspace_bytes(s), dtype=torch.uint8,
                                     device=dev)
    _run("gdr_state_space_bwd", dev, ctypes.byref(s), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
         _ptr(skip), _ptr(z), _ptr(dt_bias), _ptr(starts), _ptr(h0), _ptr(dy), _ptr(dhT),
         *(_ptr(out[n]) for n in ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "h0")),
         _ptr(workspace), _workspace_bytes(workspace, dev), _stream(stream, dev))
    _used_on(stream, dev, ws, *out.values())
    return out


def state_space_step(x, dt, A, B, C, state, *, skip=None, z=None, dt_bias=None, softplus=True,
                     y=None, stream=None):
    """One token of each sequence (``gdr_state_space_step``): x, dt, z [N, D]; B, C
    [N, G, S]; state [N, D, S] fp32 is updated in place. Returns y [N, D]."""
    s = _space_shape(x, dt, A, B, C, skip, z, dt_bias, softplus, 1)
    dev = x.device
    if state is None:
        raise ValueError("state is needed")
    _check(state, "state", F32, dev, (s.B, s.D, s.N))
    out = torch.empty_like(x, memory_format=torch.contiguous_format) if y is None else \
        _given(y, "y", x)
    _run("gdr_state_space_step", dev, ctypes.byref(s), x.data_ptr(), dt.data_ptr(), A.data_ptr(),
         B.data_ptr(), C.data_ptr(), _ptr(skip), _ptr(z), _ptr(dt_bias), state.data_ptr(),
         out.data_ptr(), _stream(stream, dev))
    if y is None and stream is not None:
        _used_on(stream, dev, out)
    return out


# ------------------------------------------------------------------ norms around a block

def _norms_inputs(x, gate, post_weight, scale, pre_weight):
    dt = _dtype(x)
    shape, dev = x.shape, x.device
    D = shape[-1]
    flat = (D,)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if gate is not None:
        _check(gate, "gate", x.dtype, dev, shape)
    _check(post_weight, "post_weight", F32, dev, flat)
    if scale is not None:
        _check(scale, "scale", F32, dev, flat)
    _check(pre_weight, "pre_weight", F32, dev, flat)
    return x.numel() // D if D else 0, D, dt


def block_norms(x, residual, post_weight, pre_weight, eps=1e-6, *, gate=None, scale=None, out=None,
                residual_out=None, stream=None):
    """The norms after and before a block (``gdr_block_norms``): r = residual + scale
    sigmoid(gate) rmsnorm(x) post_weight, y = rmsnorm(r) pre_weight, over the last axis.

    x (the block's output), residual, gate: [..., D] bf16 or fp32; post_weight, pre_weight,
    scale: [D] fp32; without gate or scale they are ones. Returns (y, r); ``residual_out``
    may be residual, x or gate itself (in place), ``out`` another of them.
    """
    rows, D, dt = _norms_inputs(x, gate, post_weight, scale, pre_weight)
    dev = x.device
    _check(residual, "residual", x.dtype, dev, x.shape)
    y = torch.empty_like(x) if out is None else _given(out, "out", x)
    r = torch.empty_like(x) if residual_out is None else _given(residual_out, "residual_out", x)
    if rows and y.data_ptr() == r.data_ptr():
        raise ValueError("out and residual_out must be apart")
    _run("gdr_block_norms", dev, rows, D, dt, x.data_ptr(), _ptr(gate), residual.data_ptr(),
         post_weight.data_ptr(), _ptr(scale), pre_weight.data_ptr(), float(eps), r.data_ptr(),
         y.data_ptr(), _stream(stream, dev))
    if stream is not None:
        _used_on(stream, dev, y if out is None else None, r if residual_out is None else None)
    return y, r


def block_norms_bwd(dy, x, sum, post_weight, pre_weight, eps=1e-6, *, gate=None, scale=None,
                    dres=None, workspace=None, stream=None):
    """Gradients of ``block_norms`` (``gdr_block_norms_bwd``): dy of y and, if given, dres of
    r = ``sum``. A dict with x, residual, gate (their dtype) and post_weight, pre_weight,
    scale (fp32; as post, pre, scale); gate and scale are None where they were not given."""
    rows, D, dt = _norms_inputs(x, gate, post_weight, scale, pre_weight)
    shape, dev, t = x.shape, x.device, x.dtype
    for v, name in ((dy, "dy"), (sum, "sum"), (dres, "dres")):
        _check(v, name, t, dev, shape)
    wide = lambda on: torch.empty(shape, dtype=t, device=dev) if on else None  # noqa: E731
    flat = lambda on: torch.empty(D, dtype=F32, device=dev) if on else None  # noqa: E731
    out = {"x": wide(True), "gate": wide(gate is not None), "residual": wide(True),
           "post": flat(True), "scale": flat(scale is not None), "pre": flat(True)}
    ws = None
    if workspace is None:
        ws = workspace = torch.empty(_bytes("gdr_block_norms_bwd_workspace", rows, D),
                                     dtype=torch.uint8, device=dev)
    _run("gdr_block_norms_bwd", dev, rows, D, dt, _ptr(dy), _ptr(dres), _ptr(x), _ptr(gate),
         _ptr(sum), _ptr(post_weight), _ptr(scale), _ptr(pre_weight), float(eps),
         *(_ptr(out[n]) for n in ("x", "gate", "residual", "post", "scale", "pre")),
         _ptr(workspace), _workspace_bytes(workspace, dev), _stream(stream, dev))
    _used_on(stream, dev, ws, *out.values())
    return out
