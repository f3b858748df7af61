"""GPU parity of the forward with bias, activation and residual in its epilogue
(slr_forward_epilogue) against the fp64 definition (oracle/epilogue.py).

Tolerances, from the arithmetic:
* Z: the products are exact in fp32 and summed in fp32, at most d_in + r + 1 of
  them, each addition within 2^-23 of the running sum (truncating adders
  included), so within (d_in + r + 1) 2^-23 B of the exact sum, B the sum of
  magnitudes; T is rounded to bf16 on the tensor-core path, 2^-8 relative, at
  most 2^-8 |T||U| in Z.
* act: its slope is at most 1.13 (gelu; silu 1.10), its fp32 evaluation within
  2^-16 |z|.
* One rounding to bf16: 2^-8 of the result (half of eps)."""
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

HALF = 2.0 ** -8   # half a bf16 step, relative


class Layer:
    """Operands of one call, host bits and fp64."""

    def __init__(self, M, d_out, d_in, r, seed, ldr=None):
        self.M, self.d_out, self.d_in, self.r = M, d_out, d_in, r
        self.X = synth.activations_bf16(M, d_in, seed, seed + 1)
        self.vals, self.meta = oracle.pack_2to4(synth.gaussian_bf16((d_out, d_in), 0.05, seed + 2))
        self.U = synth.gaussian_bf16((d_out, r), 0.1, seed + 3) if r else None
        self.V = synth.gaussian_bf16((r, d_in), 1.0 / np.sqrt(d_in), seed + 4) if r else None
        self.bias = synth.gaussian_bf16((d_out,), 0.5, seed + 5)
        self.ldr = ldr or d_out
        self.R = synth.gaussian_bf16((M, self.ldr), 1.0, seed + 6)

    def device(self):
        opt = lambda b: None if b is None else to_dev(b)  # noqa: E731
        return to_dev(self.X), to_dev(self.vals), to_dev_u8(self.meta), opt(self.U), opt(self.V)

    def reference(self, act, bias, res):
        opt = lambda b: None if b is None else bits_to_f64(b)  # noqa: E731
        S = oe.dense(self.vals, self.meta)
        return oe.forward(bits_to_f64(self.X), S, opt(self.U), opt(self.V), bits_to_f64(self.bias) if bias else None,
                          act, bits_to_f64(self.R)[:, : self.d_out] if res else None)


def check(y, z, L, act, bias, res, what):
    """y (and z where not None) within the derived tolerances of the definition."""
    Y, Z, B, BT = L.reference(act, bias, res)
    zerr = (L.d_in + L.r + 1) * 2.0 ** -23 * B + HALF * BT
    got = bits_to_f64(from_dev(y))
    err = 1.13 * zerr + 2.0 ** -16 * np.abs(Z)
    tol = err + HALF * (np.abs(Y) + err) + 1e-30
    bad = ~(np.abs(got - Y) <= tol)
    assert not bad.any(), f"{what}: Y off at {np.argwhere(bad)[0]}: {got[bad][0]} vs {Y[bad][0]}, {bad.sum()} in all"
    if z is not None:
        gz = bits_to_f64(from_dev(z))
        bad = ~(np.abs(gz - Z) <= zerr + HALF * (np.abs(Z) + zerr))
        assert not bad.any(), f"{what}: Z off at {np.argwhere(bad)[0]}"


def run(L, act="none", bias=True, res=True, pre=False, **kw):
    X, vals, meta, U, V = L.device()
    R = to_dev(L.R)[:, : L.d_out] if res else None
    Z = torch.full((L.M, L.d_out), float("nan"), dtype=torch.bfloat16, device="cuda") if pre else None
    Y = slr.forward_epilogue(X, vals, meta, U, V, bias=to_dev(L.bias) if bias else None, act=act, residual=R, preact=Z,
                             **kw)
    torch.cuda.synchronize()
    slr.check_kernel_error()
    check(Y, Z, L, act, bias, res, f"M={L.M} {L.d_out}x{L.d_in} r={L.r} {act} bias={bias} res={res} {kw}")


# Every dispatch range: streaming, split-K on 16 to 128 tokens, pair kernels.
SHAPES = [(1, 264, 256, 8), (1, 100, 128, 0), (3, 101, 384, 16), (2, 520, 256, 64), (16, 136, 512, 64),
          (17, 256, 256, 72), (33, 392, 256, 0), (64, 128, 896, 24), (65, 8, 128, 8), (130, 1032, 384, 64),
          (241, 4744, 256, 128), (300, 520, 640, 136)]


@pytest.mark.parametrize("M,d_out,d_in,r", SHAPES)
@pytest.mark.parametrize("act,bias,res,pre", [("none", True, True, False), ("gelu", True, False, True),
                                              ("silu", False, True, True)])
def test_epilogue_shapes(M, d_out, d_in, r, act, bias, res, pre):
    run(Layer(M, d_out, d_in, r, 7 * M + d_out + r), act, bias, res, pre)


@pytest.mark.parametrize("M", [1, 9, 200])
@pytest.mark.parametrize("act", oe.ACTS)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("res", [False, True])
def test_epilogue_operands(M, act, bias, res):
    run(Layer(M, 272, 256, 16, M, ldr=280), act, bias, res, pre=M != 9)


@pytest.mark.parametrize("kernel", ["small", "2sm128", "2sm240", "2sm240w"])
@pytest.mark.parametrize("M,d_out,d_in,r", [(70, 520, 256, 16), (250, 1032, 640, 64), (500, 2056, 2048, 72)])
def test_epilogue_kernels(kernel, M, d_out, d_in, r, monkeypatch):
    monkeypatch.setenv("SLR_TC_KERNEL", kernel)
    run(Layer(M, d_out, d_in, r, M + r, ldr=d_out + 24), "gelu_tanh", True, True, True, path="tensor")


@pytest.mark.parametrize("kernel", ["2smtall", "2smtallw", "2smtallk"])   # last round by tokens, whole, along K
@pytest.mark.parametrize("M,d_out,d_in,r", [(65, 264, 256, 0), (300, 1032, 512, 64), (777, 520, 1152, 8), (1000, 2056, 512, 136),
                                            (1200, 8200, 256, 64), (250, 1024, 2048, 128)])
@pytest.mark.parametrize("act,bias,res,pre", [("none", True, True, False), ("gelu", True, False, True),
                                              ("silu", False, True, True)])
def test_epilogue_in_the_512_row_kernel(kernel, M, d_out, d_in, r, act, bias, res, pre, monkeypatch):
    monkeypatch.setenv("SLR_TC_KERNEL", kernel)
    L = Layer(M, d_out, d_in, r, M + d_out + r, ldr=d_out + 16)
    run(L, act, bias, res, pre)


@pytest.mark.parametrize("kernel", ["2smtall", "2smtallk"])
def test_residual_stream_in_place_in_the_512_row_kernel(kernel, monkeypatch):
    monkeypatch.setenv("SLR_TC_KERNEL", kernel)
    L = Layer(500, 1032, 512, 64, 31)
    ops, Y = L.device(), to_dev(L.R)
    first = slr.forward_epilogue(*ops, bias=to_dev(L.bias), act="gelu_tanh", residual=to_dev(L.R))
    slr.forward_epilogue(*ops, bias=to_dev(L.bias), act="gelu_tanh", residual=Y, out=Y)
    slr.check_kernel_error()
    check(Y, None, L, "gelu_tanh", True, True, "in place")
    assert torch.equal(Y, first)


@pytest.mark.parametrize("M,path", [(1, "decode"), (5, "tensor"), (64, "tensor"), (5, "decode"), (129, "tensor"),
                                    (700, "tensor")])
def test_residual_stream_in_place(M, path):
    L = Layer(M, 1032, 512, 64, M)
    X, vals, meta, U, V = L.device()
    Y = to_dev(L.R)
    got = slr.forward_epilogue(X, vals, meta, U, V, bias=to_dev(L.bias), act="relu", residual=Y, out=Y, path=path)
    assert got.data_ptr() == Y.data_ptr()
    check(Y, None, L, "relu", True, True, f"in place M={M} {path}")


@pytest.mark.parametrize("M,d_out,path", [(1, 264, "decode"), (7, 264, "tensor"), (64, 264, "tensor"),
                                          (300, 1032, "tensor")])
def test_without_epilogue_is_the_forward(M, d_out, path):
    L = Layer(M, d_out, 256, 16, 3)
    ops = L.device()
    assert torch.equal(slr.forward_epilogue(*ops, path=path), slr.forward(*ops, path=path))


def test_chained_residual_stream():
    """Two chained layers that update one residual stream in place give the bits of ordinary calls."""
    for M in (1, 4, 33):
        L = Layer(M, 512, 512, 64, 11)
        X, vals, meta, U, V = L.device()
        b = to_dev(L.bias)
        ends = []
        for chained in (False, True):
            h, ws = to_dev(L.R), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
            for _ in range(6):
                t = slr.forward_epilogue(h, vals, meta, U, V, bias=b, act="silu", path="tensor", workspace=ws,
                                         overlap_preceding=chained)
                slr.forward_epilogue(t, vals, meta, U, V, residual=h, out=h, path="tensor", workspace=ws,
                                     overlap_preceding=chained)
            torch.cuda.synchronize()
            ends.append(h)
        slr.check_kernel_error()
        assert torch.equal(*ends)


def test_captured_call_replays():
    L = Layer(130, 1032, 384, 64, 21)
    X, vals, meta, U, V = L.device()
    R, b = to_dev(L.R), to_dev(L.bias)
    Z = torch.empty((L.M, L.d_out), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(Z)
    ws = torch.empty(slr.workspace_size(L.M, L.d_out, L.d_in, L.r), dtype=torch.uint8, device="cuda")
    call = lambda: slr.forward_epilogue(X, vals, meta, U, V, bias=b, act="gelu", residual=R, preact=Z, out=out,  # noqa: E731
                                        workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    X2 = synth.activations_bf16(L.M, L.d_in, 77, 78)
    for bits in (L.X, X2):
        X.copy_(to_dev(bits))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        if bits is L.X:
            assert torch.equal(out, first)
        L.X = bits
        check(out, Z, L, "gelu", True, True, "replayed")
    slr.check_kernel_error()


@pytest.mark.parametrize("M,path", [(1, "decode"), (6, "tensor"), (100, "tensor")])
@pytest.mark.parametrize("act", oe.ACTS)
def test_nan_and_infinity_pass(M, path, act):
    """NaN in a token's input or residual stays NaN in that token's row alone; +inf passes."""
    L = Layer(M, 264, 256, 8, 5)
    X, vals, meta, U, V = L.device()
    clean = slr.forward_epilogue(X, vals, meta, U, V, act=act, residual=to_dev(L.R), path=path)
    X[M - 1, 7] = float("nan")
    R = to_dev(L.R)
    R[0, 3] = float("inf")
    Y = slr.forward_epilogue(X, vals, meta, U, V, act=act, residual=R, path=path)
    assert torch.isnan(Y[M - 1]).all()
    if M > 1:
        assert Y[0, 3] == float("inf")
        keep = torch.ones_like(Y, dtype=torch.bool)
        keep[M - 1] = False
        keep[0, 3] = False
        assert torch.equal(Y[keep], clean[keep])


def test_second_stream_and_no_tokens():
    L = Layer(20, 264, 256, 8, 9)
    X, vals, meta, U, V = L.device()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        Y = slr.forward_epilogue(X, vals, meta, U, V, act="relu")
    s.synchronize()
    check(Y, None, L, "relu", False, False, "second stream")
    empty = slr.forward_epilogue(X[:0], vals, meta, U, V, act="relu")
    assert empty.shape == (0, 264)
