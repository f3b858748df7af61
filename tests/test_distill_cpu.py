"""CPU checks of the distillation operators: the fp64 definition's pins and the
refusals of the C ABI and the binding."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.distill as od
import sparse_rank_linear_02_b200 as slr

OK, NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, CUDA, TIMEOUT, ARG = range(9)
P = ctypes.c_void_p


def test_definition_against_closed_forms():
    # Uniform student over n columns, teacher certain of one: loss = tau^2 log n.
    loss, lse, dz, _ = od.distill(np.zeros((1, 10)), np.array([[3]]), np.array([[5.0]]), 2.0)
    assert abs(loss[0] - 4 * np.log(10)) < 1e-12 and abs(lse[0] - np.log(10)) < 1e-12
    want = np.full(10, 2.0 / 10)
    want[3] -= 2.0
    assert np.allclose(dz[0], want)
    # A teacher that lists every column with the student's own logits: nothing to learn.
    z = np.random.default_rng(0).standard_normal((2, 6))
    loss, _, dz, _ = od.distill(z, np.tile(np.arange(6), (2, 1)), z, 1.5)
    assert np.abs(loss).max() < 1e-14 and np.abs(dz).max() < 1e-14
    # Absent entries: nothing listed, columns out of range, -inf.
    for idx, t in (([[-1, 6]], [[0.0, 0.0]]), ([[1, 2]], [[-np.inf, -np.inf]])):
        loss, lse, dz, _ = od.distill(z[:1], np.array(idx), np.array(t), 1.0)
        assert loss[0] == 0 and lse[0] == 0 and not dz.any()
    # A column listed twice is a column with both entries' mass.
    a = od.distill(z[:1], np.array([[2, 2, 4]]), np.array([[0.0, 0.0, np.log(2)]]), 1.0)[2]
    b = od.distill(z[:1], np.array([[2, 4]]), np.array([[0.0, 0.0]]), 1.0)[2]
    assert np.allclose(a, b)


def test_definition_gradient_by_differences():
    rng = np.random.default_rng(1)
    z, idx, t, tau, h = rng.standard_normal((3, 9)), np.array([[0, 4, 4], [8, -1, 2], [1, 2, 3]]), rng.standard_normal((3, 3)), 0.7, 1e-6
    dz = od.distill(z, idx, t, tau)[2]
    for m in range(3):
        for v in range(9):
            e = np.zeros_like(z)
            e[m, v] = h
            num = (od.distill(z + e, idx, t, tau)[0][m] - od.distill(z - e, idx, t, tau)[0][m]) / (2 * h)
            assert abs(num - dz[m, v]) < 1e-7


def test_distill_argument_errors():
    lib = slr.lib()
    z, i, t, a, b, d = (P(0x10000 * n) for n in range(1, 7))
    f, g, s = lib.slr_distill_forward, lib.slr_distill_backward, lib.slr_distill_loss_grad
    for tau in (0.0, -1.0, 1e5, 1e-5, float("nan"), float("inf")):
        assert f(z, 2, 100, 100, i, t, 4, tau, a, b, None) == ARG
    assert f(z, -1, 100, 100, i, t, 4, 1.0, a, b, None) == SHAPE and f(z, 1 << 27, 100, 100, i, t, 4, 1.0, a, b, None) == SHAPE
    assert f(z, 2, 0, 100, i, t, 4, 1.0, a, b, None) == SHAPE and f(z, 2, 100, 99, i, t, 4, 1.0, a, b, None) == SHAPE
    assert f(z, 2, 100, 100, i, t, 0, 1.0, a, b, None) == SHAPE and f(z, 2, 100, 100, i, t, 1025, 1.0, a, b, None) == SHAPE
    assert f(None, 2, 100, 100, i, t, 4, 1.0, a, b, None) == NULL and f(z, 2, 100, 100, None, t, 4, 1.0, a, b, None) == NULL
    assert f(z, 2, 100, 100, i, None, 4, 1.0, a, b, None) == NULL and f(z, 2, 100, 100, i, t, 4, 1.0, None, b, None) == NULL
    assert f(P(0x10001), 2, 100, 100, i, t, 4, 1.0, a, b, None) == ALIGN
    assert f(z, 2, 100, 100, P(0x20002), t, 4, 1.0, a, b, None) == ALIGN
    assert f(z, 0, 100, 100, None, None, 4, 1.0, None, None, None) == OK
    assert g(z, 2, 100, 100, i, t, 4, 1.0, a, None, d, 100, None) == NULL and g(z, 2, 100, 100, i, t, 4, 1.0, None, b, d, 100, None) == NULL
    assert g(z, 2, 100, 100, i, t, 4, 1.0, a, b, None, 100, None) == NULL and g(z, 2, 100, 100, i, t, 4, 1.0, a, b, d, 99, None) == SHAPE
    assert g(z, 2, 100, 100, i, t, 4, 1.0, a, b, z, 101, None) == SHAPE          # in place with other rows
    assert s(z, 2, 100, 100, i, t, 4, 1.0, a, b, P(0x60001), 100, None) == ALIGN
    assert s(z, 2, 100, 100, i, t, 4, 1.0, None, b, d, 100, None) == NULL and s(z, 2, 100, 100, i, t, 4, 1.0, a, b, d, 99, None) == SHAPE
    assert s(z, 0, 100, 100, None, None, 4, 1.0, None, None, None, 100, None) == OK
    if not torch.cuda.is_available():
        assert f(z, 2, 100, 100, i, t, 4, 1.0, a, None, None) == DEVICE
        assert g(z, 2, 100, 100, i, t, 4, 1.0, a, b, z, 100, None) == DEVICE
        assert s(P(0x10002), 2, 100, 101, i, t, 1024, 1e4, a, b, d, 100, None) == DEVICE


def test_binding_refuses_host_tensors():
    z = torch.zeros((2, 8), dtype=torch.bfloat16)
    i, t = torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))
    with pytest.raises(ValueError, match="CUDA device"):
        slr.distill_forward(z, i, t)
