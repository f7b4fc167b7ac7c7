"""Refusals of the block operators, one argument changed at a time: every pointer of a call is an
address of its own, the call as it stands is past the check in question (its status says so), and
the change alone makes it a refusal. No call reaches a launch: its sizes need more CTAs than a grid
has, which the host finds, or its workspace is too small."""
import ctypes

import pytest
import torch

import gated_delta_rule_10_gb300 as gdr
from gated_delta_rule_10_gb300 import block

OK, INVALID, CUDA, WORKSPACE = 0, 1, 3, 4
ALL = (1 << 64) - 1              # a workspace of any size


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_10_gb300 import build
    build.build()
    return block._lib()


def conv(**kw):
    base = dict(B=65535, T=1 << 30, D=1 << 20, K=4, dtype=gdr.GDR_BF16, silu=1, x_stride=0)
    return gdr.ConvShape(**{**base, **kw})


def space(**kw):
    base = dict(B=2, T=1000, D=64, G=2, N=16, dtype=gdr.GDR_BF16, softplus=1, x_stride=0,
                dt_stride=0, z_stride=0, b_stride=0, c_stride=0)
    return gdr.StateSpaceShape(**{**base, **kw})


class Call:
    """A call by the names of its pointers, in order: `ins`, `outs` (what it writes, a state that
    it updates among them), which of them may be NULL and which need no alignment."""

    def __init__(self, call, order, outs, null=(), any_address=()):
        self.call, self.order, self.outs = call, order.split(), outs.split()
        self.null, self.any_address = null, any_address
        self.ins = [n for n in self.order if n not in self.outs]
        self.base = {n: 4096 * (i + 1) for i, n in enumerate(self.order)}

    def __call__(self, **change):
        p = {**self.base, **change}
        return self.call([p[n] for n in self.order])

    def check_pointers(self, passed):
        """`passed`: the status of the call as it stands."""
        assert self() == passed
        for n in self.order:
            assert self(**{n: None}) == (passed if n in self.null else INVALID), n
            step = 1 if n in self.any_address else 8
            assert self(**{n: self.base[n] + step}) == \
                (passed if n in self.any_address else INVALID), n

    def check_apart(self, allowed=()):
        """`allowed`: pairs that may be one buffer, which get as far as the call as it stands."""
        passed = self()
        assert passed == CUDA
        for i, o in enumerate(self.outs):
            for n in self.ins + self.outs[:i]:
                want = passed if (n, o) in allowed else INVALID
                assert self(**{o: self.base[n]}) == want, (n, o)


# a lost refusal of these calls would launch on the addresses, which are no memory
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="for machines without a GPU")


def conv_step_call(L):
    s = conv(T=1, B=(1 << 31) - 1)
    return Call(lambda p: L.gdr_short_conv_step(ctypes.byref(s), *p, None),
                "x weight bias state y", "state y", null=["bias"])


def test_conv_step_outputs_are_apart(L):
    """y and the state are no other buffer of the call."""
    conv_step_call(L).check_apart()


def space_step_call(L):
    s = space(T=1, B=(1 << 31) - 1, D=1 << 20, G=1)
    return Call(lambda p: L.gdr_state_space_step(ctypes.byref(s), *p, None),
                "x dt A B C skip z dt_bias state y", "state y", null=("skip", "z", "dt_bias"))


def test_space_step_outputs_are_apart(L):
    space_step_call(L).check_apart()


def conv_calls(L):
    s = conv()
    fwd = Call(lambda p: L.gdr_short_conv_fwd(ctypes.byref(s), *p, None),
               "x weight bias starts state y state_out", "y state_out",
               null=("bias", "starts", "state", "state_out"), any_address=("starts",))
    bwd = Call(lambda p, ws=1 << 20, n=ALL: L.gdr_short_conv_bwd(ctypes.byref(s), *p, ws, n, None),
               "x weight bias starts state dy dstate_out dx dweight dbias dstate",
               "dx dweight dbias dstate",
               null=("bias", "starts", "state", "dstate_out", "dbias", "dstate"),
               any_address=("starts",))
    return fwd, bwd


def test_conv_outputs_are_apart(L):
    for f in conv_calls(L):
        f.check_apart()


def space_calls(L, s=None):
    s = s or space()
    fwd = Call(lambda p, n=ALL: L.gdr_state_space_fwd(ctypes.byref(s), *p, 1 << 20, n, None),
               "x dt A B C skip z dt_bias starts h0 y hT", "y hT",
               null=("skip", "z", "dt_bias", "starts", "h0", "hT"), any_address=("starts",))
    bwd = Call(lambda p, n=ALL: L.gdr_state_space_bwd(ctypes.byref(s), *p, 1 << 20, n, None),
               "x dt A B C skip z dt_bias starts h0 dy dhT dx ddt dA dB dC dskip dz ddt_bias dh0",
               "dx ddt dA dB dC dskip dz ddt_bias dh0",
               null=("skip", "z", "dt_bias", "starts", "h0", "dhT", "dh0"), any_address=("starts",))
    return fwd, bwd


@no_gpu
def test_space_outputs_are_apart(L):
    """But the states of a prompt, and the gradients of them, may be one buffer."""
    fwd, bwd = space_calls(L)
    fwd.check_apart(allowed=[("h0", "hT")])
    bwd.check_apart(allowed=[("dhT", "dh0")])


def norms_calls(L, rows=100, n=ALL):
    fwd = Call(lambda p: L.gdr_block_norms(rows, 256, gdr.GDR_BF16, *p[:6], 1e-6, *p[6:], None),
               "x gate residual post scale pre sum y", "sum y", null=("gate", "scale"))
    bwd = Call(lambda p: L.gdr_block_norms_bwd(rows, 256, gdr.GDR_BF16, *p[:8], 1e-6, *p[8:],
                                               1 << 20, n, None),
               "dy dres x gate sum post scale pre dx dgate dresidual dpost dscale dpre",
               "dx dgate dresidual dpost dscale dpre", null=("dres", "gate", "scale"))
    return fwd, bwd


@no_gpu
def test_norms_outputs_are_apart(L):
    """But rows may be written over rows that are read."""
    fwd, bwd = norms_calls(L)
    fwd.check_apart(allowed=[(i, o) for i in ("x", "gate", "residual") for o in ("sum", "y")])
    bwd.check_apart(allowed=[(i, o) for i in ("dy", "dres", "x", "gate", "sum")
                             for o in ("dx", "dgate", "dresidual")])
    _, none = norms_calls(L, rows=0)         # the rows' pointers are not looked at, the weights' are
    for o, n in (("dpost", "dpre"), ("dpost", "dscale"), ("dpre", "post"), ("dscale", "scale"),
                 ("dpost", "pre")):
        assert none(**{o: none.base[n]}) == INVALID, (n, o)


# ------------------------------------------------------------------ pointers

def test_conv_pointers_one_by_one(L):
    for f in (*conv_calls(L), conv_step_call(L)):
        f.check_pointers(CUDA)


def test_space_pointers_one_by_one(L):
    """Before the workspace's size is looked at."""
    space_step_call(L).check_pointers(CUDA)
    short = lambda f: Call(lambda p: f.call(p, 16), " ".join(f.order), " ".join(f.outs),  # noqa: E731
                           f.null, f.any_address)
    fwd, bwd = space_calls(L)
    short(fwd).check_pointers(WORKSPACE)
    bwd = short(bwd)
    bwd.check_pointers(WORKSPACE)
    # a gradient is needed with what it is of
    for of, grad in (("skip", "dskip"), ("z", "dz"), ("dt_bias", "ddt_bias")):
        for bad in (None, bwd.base[grad] + 8):
            assert bwd(**{grad: bad}) == INVALID
            assert bwd(**{of: None, grad: bad}) == WORKSPACE


@no_gpu
def test_norms_pointers_one_by_one(L):
    norms_calls(L)[0].check_pointers(CUDA)


def test_norms_gradients_pointers_one_by_one(L):
    _, bwd = norms_calls(L, n=16)
    bwd.check_pointers(WORKSPACE)
    for of, grad in (("gate", "dgate"), ("scale", "dscale")):
        for bad in (None, bwd.base[grad] + 8):
            assert bwd(**{grad: bad}) == INVALID
            assert bwd(**{of: None, grad: bad}) == WORKSPACE
    # without rows only the weights' pointers are looked at
    _, none = norms_calls(L, rows=0)
    for n in ("post", "pre", "dpost", "dpre", "dscale"):
        assert none(**{n: None}) == INVALID and none(**{n: none.base[n] + 8}) == INVALID


def test_workspaces(L):
    """One byte less than asked for, none and one that is not aligned are refused."""
    n = ctypes.c_size_t()
    s = conv(B=2, T=100, D=64)
    assert L.gdr_short_conv_bwd_workspace(ctypes.byref(s), ctypes.byref(n)) == OK and n.value > 0
    p = [4096 * i for i in range(1, 12)]
    assert L.gdr_short_conv_bwd(ctypes.byref(s), *p, 1 << 20, n.value - 1, None) == WORKSPACE
    assert L.gdr_short_conv_bwd(ctypes.byref(s), *p, None, n.value, None) == WORKSPACE
    assert L.gdr_short_conv_bwd(ctypes.byref(s), *p, (1 << 20) + 4, n.value, None) == INVALID
    s = space()
    for name, count in (("fwd", 12), ("bwd", 21)):
        f = getattr(L, "gdr_state_space_" + name)
        assert getattr(L, "gdr_state_space_%s_workspace" % name)(ctypes.byref(s),
                                                                 ctypes.byref(n)) == OK
        p = [4096 * i for i in range(1, count + 1)]
        assert n.value > 0
        assert f(ctypes.byref(s), *p, 1 << 20, n.value - 1, None) == WORKSPACE
        assert f(ctypes.byref(s), *p, None, n.value, None) == WORKSPACE
        assert f(ctypes.byref(s), *p, (1 << 20) + 8, n.value, None) == INVALID
    assert L.gdr_block_norms_bwd_workspace(100, 256, ctypes.byref(n)) == OK and n.value > 0
    f = lambda ws, size: L.gdr_block_norms_bwd(  # noqa: E731
        100, 256, gdr.GDR_BF16, *range(4096, 9 * 4096, 4096), 1e-6,
        *range(9 * 4096, 15 * 4096, 4096), ws, size, None)
    assert f(1 << 20, n.value - 1) == WORKSPACE and f(None, n.value) == WORKSPACE
    assert f((1 << 20) + 4, n.value) == INVALID
