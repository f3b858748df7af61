"""CPU checks of the epilogue operators: the fp64 definitions the GPU tests
compare against, and the refusals of the C ABI and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import oracle.epilogue as oe
import synth
import sparse_rank_linear_02_b200 as slr

OK, NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, CUDA, TIMEOUT, ARG = range(9)
P = ctypes.c_void_p


@pytest.mark.parametrize("kind", oe.ACTS)
def test_slope_is_the_difference_quotient(kind):
    z = np.linspace(-9, 9, 401) + 1e-3
    h = 1e-6
    num = (oe.act(z + h, kind) - oe.act(z - h, kind)) / (2 * h)
    assert np.abs(num - oe.act_slope(z, kind)).max() < 1e-8
    assert np.abs(oe.act_slope(z, kind)).max() < 1.13   # the tests' bound on an input error's growth


def test_activation_values_against_known_points():
    assert oe.act(np.array([0.0]), "gelu")[0] == 0.0
    assert abs(oe.act(np.array([1.0]), "gelu")[0] - 0.8413447460685429) < 1e-15       # Phi(1)
    assert abs(oe.act(np.array([1.0]), "silu")[0] - 1 / (1 + np.exp(-1))) < 1e-15
    u = np.sqrt(2 / np.pi) * (1 + 0.044715)
    assert abs(oe.act(np.array([1.0]), "gelu_tanh")[0] - 0.5 * (1 + np.tanh(u))) < 1e-15
    assert list(oe.act(np.array([-2.0, 0.0, 3.0]), "relu")) == [0.0, 0.0, 3.0]


def test_dense_and_forward_agree_with_the_c_oracle():
    W = synth.gaussian_bf16((24, 64), 1.0, 1)
    vals, meta = oracle.pack_2to4(W)
    U, V, X = synth.gaussian_bf16((24, 8), 1.0, 2), synth.gaussian_bf16((8, 64), 1.0, 3), synth.gaussian_bf16((5, 64), 1.0, 4)
    f = lambda b: synth.bf16_bits_to_f32(b).astype(np.float64)  # noqa: E731
    S = oe.dense(vals, meta)
    assert np.count_nonzero(S) <= S.size // 2 and set(np.unique(S)) <= set(np.unique(f(W))) | {0.0}
    Yc, _ = oracle.forward(X, vals, meta, U, V)
    Y, Z, B, BT = oe.forward(f(X), S, f(U), f(V), None, "none", None)
    assert np.allclose(Y, Yc, rtol=1e-12, atol=1e-10) and np.all(B + 1e-9 >= np.abs(Z)) and np.all(B >= BT)


def test_input_gradient_is_the_difference_quotient():
    """<dY, Y(X)> is linear in X: with small integers its differences are exact."""
    rng = np.random.default_rng(0)
    S, U, V = rng.integers(-3, 4, (6, 8)) * 1.0, rng.integers(-2, 3, (6, 2)) * 1.0, rng.integers(-2, 3, (2, 8)) * 1.0
    X, dY = rng.integers(-3, 4, (3, 8)) * 1.0, rng.integers(-3, 4, (3, 6)) * 1.0
    dX, B, BT = oe.input_backward(dY, S, U, V)
    for m in range(3):
        for j in range(8):
            E = np.zeros_like(X)
            E[m, j] = 1.0
            up = (dY * oe.forward(X + E, S, U, V, None, "none", None)[0]).sum()
            dn = (dY * oe.forward(X - E, S, U, V, None, "none", None)[0]).sum()
            assert (up - dn) / 2 == dX[m, j]
    assert np.all(B >= np.abs(dX)) and np.all(B >= BT)


def _fwd(X=0x1000, M=16, vals=0x2000, meta=0x3000, d_out=256, d_in=256, U=0x4000, V=0x5000, r=8, bias=0x8000, act=2,
         R=0x9000, ldr=256, Z=0xa000, Y=0x6000, ws=0x7000, ws_bytes=1 << 20, path=0, flags=0):
    return slr.lib().slr_forward_epilogue(P(X), M, P(vals), P(meta), d_out, d_in, P(U), P(V), r, P(bias), act, P(R),
                                          ldr, P(Z), P(Y), P(ws), ws_bytes, path, flags, None)


def test_forward_epilogue_argument_errors():
    assert _fwd(M=0, X=0, vals=0, meta=0, Y=0) == OK
    assert _fwd(act=-1) == ARG and _fwd(act=5) == ARG
    assert _fwd(flags=2) == ARG and _fwd(path=9) == ARG
    assert _fwd(ldr=255) == SHAPE
    assert _fwd(Z=0x6000) == ARG and _fwd(Z=0x9000) == ARG   # the pre-activation in Y's or R's memory
    assert _fwd(R=0x6000, ldr=264) == SHAPE        # Y itself as residual has Y's rows
    assert _fwd(bias=0x8001) == ALIGN and _fwd(R=0x9002) == ALIGN and _fwd(Z=0xa008) == ALIGN
    assert _fwd(ldr=260) == SHAPE                  # the tensor-core path's rows of R are 16-byte aligned
    assert _fwd(X=0) == NULL and _fwd(Y=0) == NULL and _fwd(U=0) == NULL and _fwd(ws=0) == NULL
    assert _fwd(d_in=200) == SHAPE and _fwd(r=12) == SHAPE and _fwd(d_out=100, ldr=100, path=2) == SHAPE
    assert _fwd(Y=0x6008) == ALIGN and _fwd(ws_bytes=16) == WORKSPACE
    if not torch.cuda.is_available():
        assert _fwd() == DEVICE
        assert _fwd(bias=0, R=0, ldr=0, Z=0, act=0) == DEVICE
        assert _fwd(R=0x6000, ldr=256) == DEVICE   # in place
        assert _fwd(bias=0x8002) == DEVICE
        assert _fwd(M=1, ldr=260) == DEVICE and _fwd(ldr=259, path=1) == DEVICE   # one row; the streaming path


def test_binding_refuses_host_tensors_and_unknown_activations():
    X = torch.zeros((2, 128), dtype=torch.bfloat16)
    vals, meta = torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((8, 16), dtype=torch.uint8)
    with pytest.raises(ValueError, match="act one of"):
        slr.forward_epilogue(X, vals, meta, None, None, act="swish")
    with pytest.raises(ValueError, match="CUDA device"):
        slr.forward_epilogue(X, vals, meta, None, None)


def test_epilogue_backward_argument_errors():
    f = slr.lib().slr_epilogue_backward
    dy, z, dz, db = (P(0x10000 * k) for k in range(1, 5))
    assert f(dy, z, 8, 16, 5, dz, db, None) == ARG
    assert f(dy, z, 8, 16, 2, None, None, None) == NULL
    assert f(None, z, 8, 16, 2, dz, db, None) == NULL
    assert f(dy, None, 8, 16, 2, dz, db, None) == NULL
    assert f(dy, z, 8, 12, 2, dz, db, None) == SHAPE and f(dy, z, -1, 16, 2, dz, db, None) == SHAPE
    assert f(dy, z, 8, 0, 2, dz, db, None) == SHAPE and f(dy, z, 1 << 31, 16, 2, dz, db, None) == SHAPE
    assert f(P(0x10008), z, 8, 16, 2, dz, db, None) == ALIGN and f(dy, P(0x20002), 8, 16, 2, dz, db, None) == ALIGN
    assert f(dy, z, 8, 16, 2, P(0x30008), db, None) == ALIGN and f(dy, z, 8, 16, 2, dz, P(0x40004), None) == ALIGN
    if not torch.cuda.is_available():
        assert f(dy, z, 8, 16, 2, dz, None, None) == DEVICE and f(dy, None, 8, 16, 0, None, db, None) == DEVICE
        assert f(None, None, 0, 16, 2, None, db, None) == DEVICE


def test_input_backward_argument_errors_and_workspace():
    f, size = slr.lib().slr_input_backward, slr.input_backward_workspace_size
    dy, v, m, u, vv, dx, ws = (P(0x10000 * k) for k in range(1, 8))
    big = 1 << 40
    assert f(None, 0, None, None, 16, 128, None, None, 0, None, None, 0, None) == OK
    assert f(dy, -1, v, m, 16, 128, u, vv, 8, dx, ws, big, None) == SHAPE
    for d_out, d_in, r in ((12, 128, 8), (0, 128, 8), (16, 64, 8), (16, 192, 8), (16, 128, 12), (16, 128, 264)):
        assert f(dy, 4, v, m, d_out, d_in, u, vv, r, dx, ws, big, None) == SHAPE
    assert f(None, 4, v, m, 16, 128, u, vv, 8, dx, ws, big, None) == NULL and f(dy, 4, v, m, 16, 128, None, vv, 8, dx, ws, big, None) == NULL
    assert f(dy, 4, v, m, 16, 128, u, vv, 8, None, ws, big, None) == NULL and f(dy, 4, v, m, 16, 128, u, vv, 8, dx, None, big, None) == NULL
    assert f(P(0x10008), 4, v, m, 16, 128, u, vv, 8, dx, ws, big, None) == ALIGN and f(dy, 4, v, m, 16, 128, u, vv, 8, dx, P(0x70010), big, None) == ALIGN
    assert f(dy, 4, v, m, 16, 128, u, vv, 8, dx, ws, 16, None) == WORKSPACE
    assert size(0, 16, 128, 8) == 0 and size(4, 16, 128, 8) >= 4 * 8 * 2 and size(4, 16, 100, 8) == 0
    assert size(4, 16, 128, 0) == 0                                # one slice, no G
    assert size(64, 4096, 4096, 0) % (64 * 4096 * 4) == 0          # partial tiles of the slices
    if not torch.cuda.is_available():
        assert f(dy, 4, v, m, 16, 128, u, vv, 8, dx, ws, big, None) == DEVICE
        assert f(dy, 4, v, m, 16, 128, None, None, 0, dx, None, 0, None) == DEVICE
