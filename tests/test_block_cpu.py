"""Refusals of the block operators through the C ABI and the wrappers, without a GPU: every
call here fails its argument checks, which come before any CUDA call."""
import ctypes

import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from gated_delta_rule_10_gb300 import block

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
P = 4096            # an aligned address; never read
NULL = None
BIG = 1 << 60


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_10_gb300 import build
    build.build()
    return block._lib()


def conv(**kw):
    base = dict(B=2, T=100, D=64, K=4, dtype=gdr.GDR_BF16, silu=1, x_stride=0)
    return gdr.ConvShape(**{**base, **kw})


BAD_CONV = [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(D=0), INVALID), (dict(K=0), INVALID),
            (dict(dtype=5), INVALID), (dict(K=1), UNSUPPORTED), (dict(K=5), UNSUPPORTED),
            (dict(D=60), UNSUPPORTED), (dict(D=(1 << 20) + 8), UNSUPPORTED),
            (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
            (dict(x_stride=56), INVALID), (dict(x_stride=68), INVALID), (dict(x_stride=-64), INVALID),
            (dict(x_stride=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("change,want", BAD_CONV, ids=str)
def test_conv_shapes(L, change, want):
    s = ctypes.byref(conv(**change))
    n = ctypes.c_size_t()
    assert L.gdr_short_conv_bwd_workspace(s, ctypes.byref(n)) == want
    assert L.gdr_short_conv_fwd(s, P, P, P, P, P, P, 2 * P, NULL) == want
    assert L.gdr_short_conv_bwd(s, *[P] * 7, *[2 * P] * 5, BIG, NULL) == want


def test_conv_pointers(L):
    s = ctypes.byref(conv())
    base = [P, P, P, P, P, P, 2 * P]                 # x weight bias starts state y state_out
    for i in (0, 1, 5):
        bad = list(base)
        bad[i] = NULL
        assert L.gdr_short_conv_fwd(s, *bad, NULL) == INVALID
    for i in (0, 1, 2, 4, 5, 6):
        bad = list(base)
        bad[i] = P + 8
        assert L.gdr_short_conv_fwd(s, *bad, NULL) == INVALID
    base[6] = P                                      # a state is not updated in place
    assert L.gdr_short_conv_fwd(s, *base, NULL) == INVALID
    n = ctypes.c_size_t()
    assert L.gdr_short_conv_bwd_workspace(s, ctypes.byref(n)) == OK and n.value > 0
    assert L.gdr_short_conv_bwd_workspace(s, NULL) == INVALID
    assert L.gdr_short_conv_bwd_workspace(NULL, ctypes.byref(n)) == INVALID
    back = [P] * 7 + [2 * P] * 4     # x weight bias starts state dy dstate_out dx dw dbias dstate
    for i in (0, 1, 5, 7, 8):
        bad = list(back)
        bad[i] = NULL
        assert L.gdr_short_conv_bwd(s, *bad, P, n.value, NULL) == INVALID
    assert L.gdr_short_conv_bwd(s, *back, P, n.value - 1, NULL) == WORKSPACE
    assert L.gdr_short_conv_bwd(s, *back, NULL, n.value, NULL) == WORKSPACE
    assert L.gdr_short_conv_bwd(s, *back, P + 4, n.value, NULL) == INVALID
    back[10] = P
    assert L.gdr_short_conv_bwd(s, *back, P, n.value, NULL) == INVALID


def test_conv_step(L):
    step = lambda s, p: L.gdr_short_conv_step(ctypes.byref(s), *p, NULL)  # noqa: E731
    assert step(conv(), [P] * 5) == INVALID                              # T = 100
    for i in (0, 1, 3, 4):                           # x weight bias state y
        bad = [P] * 5
        bad[i] = NULL
        assert step(conv(T=1), bad) == INVALID


def space(**kw):
    base = dict(B=2, T=100, D=64, G=2, N=16, dtype=gdr.GDR_BF16, softplus=1, x_stride=0,
                dt_stride=0, z_stride=0, b_stride=0, c_stride=0)
    return gdr.StateSpaceShape(**{**base, **kw})


BAD_SPACE = [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(D=0), INVALID), (dict(G=0), INVALID),
             (dict(N=0), INVALID), (dict(G=3), INVALID), (dict(dtype=2), INVALID),
             (dict(N=4), UNSUPPORTED), (dict(N=24), UNSUPPORTED), (dict(N=128), UNSUPPORTED),
             (dict(G=16), UNSUPPORTED), (dict(D=1 << 21), UNSUPPORTED),
             (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
             (dict(x_stride=63), INVALID), (dict(dt_stride=68), INVALID), (dict(z_stride=8), INVALID),
             (dict(b_stride=24), INVALID), (dict(c_stride=36), INVALID),
             (dict(c_stride=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("change,want", BAD_SPACE, ids=str)
def test_space_shapes(L, change, want):
    s = ctypes.byref(space(**change))
    n = ctypes.c_size_t()
    assert L.gdr_state_space_fwd_workspace(s, ctypes.byref(n)) == want
    assert L.gdr_state_space_bwd_workspace(s, ctypes.byref(n)) == want
    assert L.gdr_state_space_fwd(s, *[P] * 13, BIG, NULL) == want
    assert L.gdr_state_space_bwd(s, *[P] * 22, BIG, NULL) == want


def test_space_pointers(L):
    s = ctypes.byref(space(T=1000))          # cut into segments
    n = ctypes.c_size_t()
    assert L.gdr_state_space_fwd_workspace(s, ctypes.byref(n)) == OK and n.value > 0
    # x dt A B C skip z dt_bias starts h0 y hT
    fwd = lambda p, ws=P, size=BIG: L.gdr_state_space_fwd(s, *p, ws, size, NULL)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 10):
        bad = [P] * 12
        bad[i] = NULL
        assert fwd(bad) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10, 11):
        bad = [P] * 12
        bad[i] = P + 8
        assert fwd(bad) == INVALID
    assert fwd([P] * 12, P, n.value - 1) == WORKSPACE
    assert fwd([P] * 12, NULL) == WORKSPACE
    assert fwd([P] * 12, P + 4) == INVALID
    full = space(B=64, D=8192, G=1)          # fills the GPU: none
    assert L.gdr_state_space_fwd_workspace(ctypes.byref(full), ctypes.byref(n)) == OK
    assert n.value == 0
    assert L.gdr_state_space_bwd_workspace(s, ctypes.byref(n)) == OK and n.value > 0
    assert L.gdr_state_space_bwd_workspace(s, NULL) == INVALID
    # x dt A B C skip z dt_bias starts h0 dy dhT | dx ddt dA dB dC dskip dz ddt_bias dh0
    bwd = lambda p, ws=P, size=BIG: L.gdr_state_space_bwd(s, *p, ws, size, NULL)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 10, 12, 13, 14, 15, 16, 17, 18, 19):
        bad = [P] * 21
        bad[i] = NULL
        assert bwd(bad) == INVALID, i
    assert bwd([P] * 21, P, n.value - 1) == WORKSPACE
    assert bwd([P] * 21, P + 8) == INVALID


def test_space_segments_grow_with_the_sequence(L):
    """Room for the kept states, one per 16 tokens, and no more segments than tiles."""
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    for T in (1, 16, 17, 5000):
        s = space(T=T, B=1, G=1)
        assert L.gdr_state_space_fwd_workspace(ctypes.byref(s), ctypes.byref(n)) == OK
        assert L.gdr_state_space_bwd_workspace(ctypes.byref(s), ctypes.byref(m)) == OK
        assert (n.value == 0) == (T <= 32)
        assert m.value >= -(-T // 16) * 64 * 16 * 4


def test_space_step(L):
    step = lambda s, p: L.gdr_state_space_step(ctypes.byref(s), *p, NULL)  # noqa: E731
    assert step(space(), [P] * 10) == INVALID
    for i in (0, 1, 2, 3, 4, 8, 9):          # x dt A B C skip z dt_bias state y
        bad = [P] * 10
        bad[i] = NULL
        assert step(space(T=1), bad) == INVALID


def test_norms(L):
    f = lambda rows, D, dt=gdr.GDR_BF16, eps=1e-6, p=(P, P, P, P, P, P, P, 2 * P): (  # noqa: E731
        L.gdr_block_norms(rows, D, dt, *p[:6], eps, *p[6:], NULL))
    assert f(-1, 64) == INVALID and f(4, 0) == INVALID and f(4, 64, 9) == INVALID
    assert f(4, 64, eps=-1.0) == INVALID and f(4, 64, eps=float("nan")) == INVALID
    assert f(4, 60) == UNSUPPORTED and f(4, 8200) == UNSUPPORTED and f(1 << 31, 64) == UNSUPPORTED
    assert f(0, 64, p=(NULL,) * 8) == OK
    good = [P, P, P, P, P, P, P, 2 * P]      # x gate residual post scale pre sum y
    for i in (0, 2, 3, 5, 6, 7):
        bad = list(good)
        bad[i] = NULL
        assert f(4, 64, p=bad) == INVALID
    for i in range(8):
        bad = list(good)
        bad[i] = P + 8
        assert f(4, 64, p=bad) == INVALID
    assert f(4, 64, p=[P] * 8) == INVALID    # the sum and y are apart
    n = ctypes.c_size_t()
    assert L.gdr_block_norms_bwd_workspace(100, 256, ctypes.byref(n)) == OK and n.value > 0
    assert L.gdr_block_norms_bwd_workspace(100, 250, ctypes.byref(n)) == UNSUPPORTED
    assert L.gdr_block_norms_bwd_workspace(100, 256, NULL) == INVALID
    # dy dres x gate sum post scale pre | dx dgate dres dpost dscale dpre
    ins, outs = [P] * 8, [2 * P, 3 * P, 4 * P, P, P, P]
    bwd = lambda i, o, ws=P, size=BIG: L.gdr_block_norms_bwd(  # noqa: E731
        100, 256, gdr.GDR_BF16, *i, 1e-6, *o, ws, size, NULL)
    for k in (0, 2, 4, 5, 7):
        bad = list(ins)
        bad[k] = NULL
        assert bwd(bad, outs) == INVALID
    for k in range(6):
        bad = list(outs)
        bad[k] = NULL
        assert bwd(ins, bad) == INVALID
    assert bwd(ins, [P, P, 2 * P, P, P, P]) == INVALID
    assert bwd(ins, outs, P, n.value - 1) == WORKSPACE and bwd(ins, outs, NULL) == WORKSPACE
    assert bwd(ins, outs, P + 4) == INVALID


def test_outputs_are_apart(L):
    """An output that is an input's or another output's buffer is refused, whichever it is."""
    s = ctypes.byref(conv())
    ins, outs = [P * i for i in range(1, 6)], [P * i for i in (6, 7)]
    for o in range(2):
        for i in (0, 4):                             # x, state
            bad = list(outs)
            bad[o] = ins[i]
            assert L.gdr_short_conv_fwd(s, *ins, *bad, NULL) == INVALID
    assert L.gdr_short_conv_fwd(s, *ins, outs[0], outs[0], NULL) == INVALID
    # x weight bias starts state dy dstate_out | dx dweight dbias dstate
    ins, outs = [P * i for i in range(1, 8)], [P * i for i in range(8, 12)]
    for o in range(4):
        for i in (0, 1, 2, 4, 5, 6):
            bad = list(outs)
            bad[o] = ins[i]
            assert L.gdr_short_conv_bwd(s, *ins, *bad, 99 * P, BIG, NULL) == INVALID
        bad = list(outs)
        bad[o] = outs[o - 1]
        assert L.gdr_short_conv_bwd(s, *ins, *bad, 99 * P, BIG, NULL) == INVALID
    s = ctypes.byref(space())
    # x dt A B C skip z dt_bias starts h0 | y hT
    ins, outs = [P * i for i in range(1, 11)], [P * i for i in (11, 12)]
    for i in (0, 1, 3, 4, 6, 9):
        assert L.gdr_state_space_fwd(s, *ins, ins[i], outs[1], 99 * P, BIG, NULL) == INVALID
    for i in (0, 1, 2, 3, 4, 6):
        assert L.gdr_state_space_fwd(s, *ins, outs[0], ins[i], 99 * P, BIG, NULL) == INVALID
    assert L.gdr_state_space_fwd(s, *ins, outs[0], outs[0], 99 * P, BIG, NULL) == INVALID
    # x dt A B C skip z dt_bias starts h0 dy dhT | dx ddt dA dB dC dskip dz ddt_bias dh0
    ins, outs = [P * i for i in range(1, 13)], [P * i for i in range(13, 22)]
    for o in range(9):
        for i in (0, 1, 2, 3, 4, 5, 6, 7, 9, 10):
            bad = list(outs)
            bad[o] = ins[i]
            assert L.gdr_state_space_bwd(s, *ins, *bad, 99 * P, BIG, NULL) == INVALID
        bad = list(outs)
        bad[o] = outs[o - 1]
        assert L.gdr_state_space_bwd(s, *ins, *bad, 99 * P, BIG, NULL) == INVALID


def test_python_refusals():
    """The wrappers name the argument; tensors on the CPU are refused."""
    x, w = torch.zeros(1, 8, 64), torch.zeros(64, 4)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.short_conv_fwd(x, w)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        gdr.short_conv_fwd(x.half(), w)
    with pytest.raises(ValueError, match=r"\[B, T, D\]"):
        gdr.short_conv_fwd(x[0], w)
    with pytest.raises(ValueError, match="channels"):
        gdr.short_conv_bwd(x, x, w[:32])
    with pytest.raises(ValueError, match=r"\[N, D\]"):
        gdr.short_conv_step(x, w, None, x)
    A, B = torch.zeros(64, 16), torch.zeros(1, 8, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.state_space_fwd(x, x, A, B, B)
    with pytest.raises(ValueError, match="G, N"):
        gdr.state_space_fwd(x, x, A, B[:, :, 0], B)
    with pytest.raises(ValueError, match="channels"):
        gdr.state_space_bwd(x, x, x, A[:32], B, B)
    with pytest.raises(ValueError, match=r"\[N, D\]"):
        gdr.state_space_step(x, x, A, B, B, A)
    with pytest.raises(ValueError):
        gdr.block_norms(x, x, torch.zeros(64), torch.zeros(64))
    with pytest.raises(ValueError, match="starts"):
        block._starts(torch.zeros(1, 8), torch.device("cuda", 0), (1, 8))
