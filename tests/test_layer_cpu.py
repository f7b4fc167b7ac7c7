"""Refusals of the layer operators through the C ABI, without a GPU: every call here
fails its argument checks, which come before any CUDA call."""
import ctypes

import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from gated_delta_rule_10_gb300 import layer

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
P = 4096            # an aligned address; never read
NULL = None


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_10_gb300 import build
    build.build()
    return layer._lib()


def shape(**kw):
    base = dict(B=2, T=100, H=4, Hk=2, dk=64, dv=128, dtype=gdr.GDR_BF16, decay_per_head=0,
                scale=0.1, q_stride=0, k_stride=0, v_stride=0)
    return layer.DecayShape(**{**base, **kw})


BAD_SHAPES = [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
              (dict(Hk=3), INVALID), (dict(dtype=7), INVALID), (dict(scale=float("nan")), INVALID),
              (dict(dk=32), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(dk=-64), INVALID),
              (dict(q_stride=64), INVALID), (dict(k_stride=132), INVALID),
              (dict(v_stride=-512), INVALID), (dict(v_stride=1 << 31), UNSUPPORTED),
              (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(B=40000), UNSUPPORTED)]


@pytest.mark.parametrize("change,want", BAD_SHAPES, ids=lambda c: str(c))
def test_decay_shapes(L, change, want):
    s = ctypes.byref(shape(**change))
    n = ctypes.c_size_t()
    assert L.gdr_decay_chunk_fwd_workspace(s, ctypes.byref(n)) == want
    assert L.gdr_decay_chunk_bwd_workspace(s, ctypes.byref(n)) == want
    assert L.gdr_decay_chunk_fwd(s, *[P] * 8, 1 << 40, NULL) == want
    assert L.gdr_decay_chunk_bwd(s, *[P] * 13, 1 << 40, NULL) == want


@pytest.mark.parametrize("null", [0, 1, 2, 3, 5])
def test_decay_forward_pointers(L, null):
    args = [P] * 8                       # q k v g h0 o hT workspace
    args[null] = NULL
    assert L.gdr_decay_chunk_fwd(ctypes.byref(shape()), *args, 1 << 40, NULL) == INVALID
    args[null] = P + 8 if null != 3 else P + 2
    assert L.gdr_decay_chunk_fwd(ctypes.byref(shape()), *args, 1 << 40, NULL) == INVALID


@pytest.mark.parametrize("null", [0, 1, 2, 3, 5, 7, 8, 9, 10])
def test_decay_backward_pointers(L, null):
    args = [P] * 13                      # q k v g h0 dO dhT dq dk dv dg dh0 workspace
    args[null] = NULL
    assert L.gdr_decay_chunk_bwd(ctypes.byref(shape()), *args, 1 << 40, NULL) == INVALID


def test_decay_workspaces(L):
    n = ctypes.c_size_t()
    few = shape(B=1, T=5000)             # cut into segments: their states
    assert L.gdr_decay_chunk_fwd_workspace(ctypes.byref(few), ctypes.byref(n)) == OK
    assert n.value > 0
    args = [P] * 8
    assert L.gdr_decay_chunk_fwd(ctypes.byref(few), *args, n.value - 1, NULL) == WORKSPACE
    args[7] = NULL
    assert L.gdr_decay_chunk_fwd(ctypes.byref(few), *args, n.value, NULL) == WORKSPACE
    args[7] = P + 4
    assert L.gdr_decay_chunk_fwd(ctypes.byref(few), *args, n.value, NULL) == INVALID
    many = shape(B=64, H=8, Hk=8)        # fills the GPU: none
    assert L.gdr_decay_chunk_fwd_workspace(ctypes.byref(many), ctypes.byref(n)) == OK
    assert n.value == 0
    assert L.gdr_decay_chunk_bwd_workspace(ctypes.byref(many), ctypes.byref(n)) == OK
    assert n.value > 0
    assert L.gdr_decay_chunk_bwd(ctypes.byref(many), *[P] * 13, n.value - 1, NULL) == WORKSPACE
    assert L.gdr_decay_chunk_fwd_workspace(ctypes.byref(many), NULL) == INVALID
    assert L.gdr_decay_chunk_fwd_workspace(NULL, ctypes.byref(n)) == INVALID


def test_decay_workspace_grows_with_the_sequence_and_bounds_a_segment(L):
    n = ctypes.c_size_t()
    sizes = []
    for T in (1, 4096, 4097, 100000):
        s = shape(B=64, H=8, Hk=8, T=T)
        assert L.gdr_decay_chunk_bwd_workspace(ctypes.byref(s), ctypes.byref(n)) == OK
        sizes.append(n.value)
    assert sizes == sorted(sizes)


def test_step(L):
    args = [P] * 6                       # q k v g state o
    assert L.gdr_decay_step(ctypes.byref(shape()), *args, NULL) == INVALID      # T = 100
    one = shape(T=1)
    for i in range(6):
        bad = list(args)
        bad[i] = NULL
        assert L.gdr_decay_step(ctypes.byref(one), *bad, NULL) == INVALID
    assert L.gdr_decay_step(ctypes.byref(shape(T=1, B=1 << 30)), *args, NULL) == UNSUPPORTED


def test_norm(L):
    f = lambda rows, D, dt=gdr.GDR_BF16, eps=1e-6, p=(P,) * 5: L.gdr_add_rmsnorm(  # noqa: E731
        rows, D, dt, p[0], p[1], p[2], eps, p[3], p[4], NULL)
    assert f(-1, 64) == INVALID and f(4, 0) == INVALID and f(4, 64, 9) == INVALID
    assert f(4, 64, eps=-1.0) == INVALID and f(4, 64, eps=float("inf")) == INVALID
    assert f(4, 60) == UNSUPPORTED and f(4, 8200) == UNSUPPORTED and f(1 << 31, 64) == UNSUPPORTED
    assert f(0, 64, p=(NULL,) * 5) == OK
    for i in range(5):
        p = [P] * 5
        p[i] = NULL
        assert f(4, 64, p=p) == INVALID
        p[i] = P + 8
        assert f(4, 64, p=p) == INVALID
    assert L.gdr_add_rmsnorm_fp8(4, 64, gdr.GDR_BF16, P, P, P, 1e-6, P, P, NULL, NULL) == INVALID
    n = ctypes.c_size_t()
    assert L.gdr_add_rmsnorm_bwd_workspace(100, 256, ctypes.byref(n)) == OK and n.value > 0
    bwd = lambda ws, size: L.gdr_add_rmsnorm_bwd(100, 256, gdr.GDR_BF16, P, P, P, 1e-6, NULL, P, P,  # noqa: E731
                                                 ws, size, NULL)
    assert bwd(NULL, n.value) == WORKSPACE and bwd(P, n.value - 1) == WORKSPACE
    assert bwd(P + 4, n.value) == INVALID
    assert L.gdr_add_rmsnorm_bwd_workspace(100, 250, ctypes.byref(n)) == UNSUPPORTED


def rot(**kw):
    base = dict(B=2, T=3, H=4, Hk=2, d=64, rot=32, dtype=gdr.GDR_BF16, interleaved=0, inverse=0,
                start=0, table_length=100, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0)
    return layer.RotaryShape(**{**base, **kw})


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), INVALID), (dict(H=0, Hk=0), INVALID), (dict(rot=8), INVALID),
    (dict(rot=40), INVALID), (dict(rot=80), INVALID), (dict(d=72, rot=32), UNSUPPORTED),
    (dict(table_length=0), INVALID), (dict(dtype=3), INVALID), (dict(q_stride=255), INVALID),
    (dict(q_out_stride=260), INVALID), (dict(T=1 << 30), UNSUPPORTED)])
def test_rotary_shapes(L, change, want):
    assert L.gdr_rotary(ctypes.byref(rot(**change)), *[P] * 7, NULL) == want


def test_rotary_pointers_and_tables(L):
    for i in (0, 1, 2, 3, 5, 6):         # q k cos sin pos q_out k_out
        args = [P] * 7
        args[i] = NULL
        assert L.gdr_rotary(ctypes.byref(rot()), *args, NULL) == INVALID
        args[i] = P + 8
        assert L.gdr_rotary(ctypes.byref(rot()), *args, NULL) == INVALID
    assert L.gdr_rotary(ctypes.byref(rot(T=0)), *[NULL] * 7, NULL) == OK
    z = layer.RotaryScaling(0, 1.0, 0, 32.0, 1.0, 1.0)
    t = lambda n, r, base, s: L.gdr_rotary_table(n, r, base, ctypes.byref(s), P, P, NULL)  # noqa: E731
    assert t(0, 32, 1e4, z) == INVALID and t(8, 24, 1e4, z) == INVALID and t(8, 32, 1.0, z) == INVALID
    for bad in (layer.RotaryScaling(4, 2.0, 0, 32.0, 1.0, 1.0), layer.RotaryScaling(1, 0.5, 0, 0, 0, 0),
                layer.RotaryScaling(3, 2.0, 0, 32.0, 1.0, 1.0),
                layer.RotaryScaling(3, 2.0, 64, 1.0, 1.0, 1.0),
                layer.RotaryScaling(3, 2.0, 64, 32.0, 1.0, 0.0)):
        assert t(8, 32, 1e4, bad) == INVALID


def test_python_refusals():
    """The wrappers name the argument; tensors on the CPU are refused."""
    q = torch.zeros(1, 8, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.decay_chunk_fwd(q, q, q, torch.zeros(1, 8, 2))
    with pytest.raises(ValueError, match="bf16 or fp32"):
        gdr.decay_chunk_fwd(q.half(), q.half(), q.half(), torch.zeros(1, 8, 2))
    with pytest.raises(ValueError):
        gdr.add_rmsnorm(torch.zeros(2, 64), torch.zeros(2, 64), torch.zeros(64))
    with pytest.raises(ValueError):
        gdr.rotary(q, q, torch.zeros(8, 32), torch.zeros(8, 32))
    with pytest.raises(ValueError, match="scaling"):
        gdr.rotary_table(8, 32, scaling="other", device="cpu")
