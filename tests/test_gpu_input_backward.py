"""GPU parity of the gradient of the layer's input (slr_input_backward):
dX = dY S + (dY U) V against the fp64 definition (oracle/epilogue.py).

Tolerance, from the arithmetic: the products are exact in fp32 and summed in fp32,
at most d_out + r of them (and eight partial tiles), each addition within 2^-23
of the sum of magnitudes B so far; G = dY U is rounded to bf16, 2^-8 relative, at
most 2^-8 |dY||U||V| in dX, and carries its own sum's error; one rounding to bf16."""
import numpy as np
import pytest
import torch

import oracle
import oracle.epilogue as oe
import synth
from gpu_util import bits_to_f64, from_dev, to_dev, to_dev_u8

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_rank_linear_02_b200 as slr


class Problem:
    def __init__(self, M, d_out, d_in, r, seed):
        self.shape = (M, d_out, d_in, r)
        self.dY = synth.gaussian_bf16((M, d_out), 1.0, seed)
        self.vals, self.meta = oracle.pack_2to4(synth.gaussian_bf16((d_out, d_in), 0.05, seed + 1))
        self.U = synth.gaussian_bf16((d_out, r), 0.1, seed + 2) if r else None
        self.V = synth.gaussian_bf16((r, d_in), 0.1, seed + 3) if r else None

    def device(self):
        opt = lambda b: None if b is None else to_dev(b)  # noqa: E731
        return to_dev(self.dY), to_dev(self.vals), to_dev_u8(self.meta), opt(self.U), opt(self.V)

    def check(self, dX, what=""):
        M, d_out, d_in, r = self.shape
        opt = lambda b: None if b is None else bits_to_f64(b)  # noqa: E731
        want, B, BT = oe.input_backward(bits_to_f64(self.dY), oe.dense(self.vals, self.meta), opt(self.U), opt(self.V))
        got = bits_to_f64(from_dev(dX))
        err = (2 * d_out + r + 8) * 2.0 ** -23 * B + 2.0 ** -8 * BT
        bad = ~(np.abs(got - want) <= err + 2.0 ** -8 * (np.abs(want) + err))
        assert not bad.any(), f"{what} {self.shape}: off at {np.argwhere(bad)[0]}: {got[bad][0]} vs {want[bad][0]}, {bad.sum()} in all"


@pytest.mark.parametrize("halves", ["1", "2"])   # tiles of one or two 256-column halves
@pytest.mark.parametrize("M,d_out,d_in,r", [(1, 8, 128, 0), (1, 64, 128, 8), (5, 72, 256, 0), (16, 256, 256, 64),
                                            (17, 520, 384, 72), (64, 4096, 512, 64), (100, 1032, 640, 136),
                                            (241, 264, 1152, 256), (300, 2056, 896, 16), (500, 136, 4096, 128),
                                            (1000, 1000, 2048, 8), (33, 14336, 256, 64),
                                            (960, 200, 640, 192), (2100, 328, 1408, 24)])
def test_input_backward(M, d_out, d_in, r, halves, monkeypatch):
    monkeypatch.setenv("SLR_DX_HALVES", halves)
    p = Problem(M, d_out, d_in, r, M + d_out + d_in + r)
    dX = slr.input_backward(*p.device())
    torch.cuda.synchronize()
    slr.check_kernel_error()
    p.check(dX)


def test_full_size_layer():
    p = Problem(2048, 14336, 4096, 64, 5)
    dX = slr.input_backward(*p.device())
    slr.check_kernel_error()
    M, d_out, d_in, r = p.shape
    # Against a product of the same operands in fp64 on the device (the host's takes minutes).
    S = torch.from_numpy(oe.dense(p.vals, p.meta)).cuda()
    dY, U, V = (torch.from_numpy(bits_to_f64(b)).cuda() for b in (p.dY, p.U, p.V))
    want, B = dY @ S + (dY @ U) @ V, dY.abs() @ S.abs()
    BT = (dY.abs() @ U.abs()) @ V.abs()
    err = (2 * d_out + r + 8) * 2.0 ** -23 * (B + BT) + 2.0 ** -8 * BT
    assert bool(((dX.double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all())
    assert float((dX.double() - want).norm() / want.norm()) <= 5e-3
    assert torch.equal(dX, slr.input_backward(*p.device()))


def test_what_lies_behind_and_empty_batch():
    p = Problem(37, 264, 384, 24, 3)
    ops = p.device()
    out = torch.full((40, 384), 7.0, dtype=torch.bfloat16, device="cuda")
    slr.input_backward(*ops, out=out[:37])
    torch.cuda.synchronize()
    p.check(out[:37])
    assert torch.all(out[37:] == 7.0)
    assert slr.input_backward(ops[0][:0], *ops[1:]).shape == (0, 384)


@pytest.mark.parametrize("halves", ["1", "2"])
def test_zero_and_nan_rows(halves, monkeypatch):
    monkeypatch.setenv("SLR_DX_HALVES", halves)
    p = Problem(50, 520, 256, 16, 9)
    dY, vals, meta, U, V = p.device()
    clean = slr.input_backward(dY, vals, meta, U, V)
    dY[3] = 0
    dY[20, 11] = float("nan")
    dX = slr.input_backward(dY, vals, meta, U, V)
    assert torch.count_nonzero(dX[3]) == 0 and torch.isnan(dX[20]).all()
    keep = [i for i in range(50) if i not in (3, 20)]
    assert torch.equal(dX[keep], clean[keep])


@pytest.mark.parametrize("M,d_out", [(64, 4096), (300, 520)])
def test_captured_and_second_stream(M, d_out):
    p = Problem(M, d_out, 512, 64, 11)
    ops = p.device()
    first = slr.input_backward(*ops)
    ws = torch.empty(max(slr.input_backward_workspace_size(M, d_out, 512, 64), 256), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):   # one workspace, calls in a row
            slr.input_backward(*ops, out=out, workspace=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = slr.input_backward(*ops)
    s.synchronize()
    assert torch.equal(other, first)
    slr.check_kernel_error()


def test_gradient_by_differences():
    """<dY, forward(X)> is linear in X: a step along one column of X moves it by
    the column of dX, up to the rounding of both."""
    M, d_out, d_in, r = 64, 264, 256, 16
    p = Problem(M, d_out, d_in, r, 21)
    dY, vals, meta, U, V = p.device()
    dX = slr.input_backward(dY, vals, meta, U, V).double()
    X = torch.zeros((M, d_in), dtype=torch.bfloat16, device="cuda")
    for col in (0, 77, 255):
        X.zero_()
        X[:, col] = 1.0
        Y = slr.forward(X, vals, meta, U, V, path="tensor").double()
        num = (dY.double() * Y).sum(1)
        tol = 2.0 ** -7 * (dY.double().abs() * Y.abs()).sum(1) + 2.0 ** -7 * (
            dY.double().abs() @ U.double().abs() @ V.double().abs())[:, col] + 2.0 ** -8 * dX[:, col].abs()
        assert bool(((dX[:, col] - num).abs() <= tol).all())
