"""Argument checks of the epilogue's entry points: an empty batch looks at no
pointer, nulls come before sizes and sizes before alignment, and an operand that
is not looked at is not checked."""
import ctypes

import pytest
import torch

import sparse_rank_linear_02_b200 as slr
from test_epilogue_cpu import _fwd

OK, NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, CUDA, TIMEOUT, ARG = range(9)
P = ctypes.c_void_p


@pytest.mark.parametrize("kw", [dict(R=0x9002), dict(Z=0xa008), dict(bias=0x8001), dict(Z=0x6000), dict(Z=0x9000),
                                dict(ldr=0), dict(ldr=260), dict(R=0x6000, ldr=264), dict(ws=0, ws_bytes=0)])
def test_forward_epilogue_of_no_tokens_looks_at_no_operand(kw):
    assert _fwd(M=0, **kw) == OK
    assert _fwd(M=0, X=0, vals=0, meta=0, U=0, V=0, **{**dict(Y=0), **kw}) == OK


def test_forward_epilogue_of_no_tokens_still_refuses_what_no_call_means():
    assert _fwd(M=0, act=9) == ARG and _fwd(M=0, flags=2) == ARG and _fwd(M=0, path=7) == ARG
    assert _fwd(M=-1) == SHAPE and _fwd(M=0, r=-8) == SHAPE


def test_forward_epilogue_checks_in_order():
    assert _fwd(X=0, ldr=255) == NULL and _fwd(Y=0, R=0x9002) == NULL and _fwd(ws=0, bias=0x8001) == NULL
    assert _fwd(ldr=255, R=0x9002) == SHAPE and _fwd(ldr=260, Z=0xa008) == SHAPE and _fwd(d_in=200, R=0x9002) == SHAPE
    assert _fwd(R=0x9002, ws_bytes=16) == ALIGN and _fwd(Z=0xa008, ws_bytes=16) == ALIGN
    assert _fwd(bias=0x8001, ws_bytes=16) == ALIGN
    assert _fwd(Z=0x6000, ldr=255) == ARG and _fwd(Z=0x9000, ws_bytes=16) == ARG   # arguments that never go together
    assert _fwd(ws_bytes=16) == WORKSPACE


def test_epilogue_backward_without_an_activation_does_not_look_at_z():
    f = slr.lib().slr_epilogue_backward
    dy, dz, db = (P(0x10000 * k) for k in (1, 3, 4))
    if not torch.cuda.is_available():
        assert f(dy, P(0x20002), 8, 16, 0, dz, db, None) == DEVICE
    assert f(dy, P(0x20002), 8, 16, 1, dz, db, None) == ALIGN
