"""GPU parity of the gradient through the epilogue (slr_epilogue_backward):
dZ = dY act'(Z), db = the column sums of dZ, against the fp64 definition
(oracle/epilogue.py).

Tolerances, from the arithmetic: the fp32 slope is within 2^-16 of the exact
one (its exponentials and quotients carry a few 2^-22 relative, times at most
|z| (1 + 0.14 z^2) sigma (1 - sigma) < 10 in the tanh form); one rounding of dZ
to bf16 (2^-8 relative); db adds unrounded products in fp32 in chains of at
most 64 rows, M / 64 of those, then at most 32 + 8, each addition within 2^-24
of a partial sum that the sum of magnitudes bounds."""
import numpy as np
import pytest
import torch

import oracle.epilogue as oe
import synth
from gpu_util import bits_to_f64, from_dev, to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_rank_linear_02_b200 as slr


def check(dZ, db, dY, Z, act, what):
    g, z = bits_to_f64(dY), bits_to_f64(Z)
    want = g * oe.act_slope(z, act)
    if dZ is not None:
        err = np.abs(g) * 2.0 ** -16
        bad = ~(np.abs(bits_to_f64(from_dev(dZ)) - want) <= err + 2.0 ** -8 * (np.abs(want) + err) + 1e-38)
        assert not bad.any(), f"{what}: dZ off at {np.argwhere(bad)[0]}"
    if db is not None:
        M = g.shape[0]
        tol = np.abs(g).sum(0) * (2.0 ** -16 + (104 + M / 64) * 2.0 ** -24 * 1.13) + 1e-38
        bad = ~(np.abs(db.double().cpu().numpy() - want.sum(0)) <= tol)
        assert not bad.any(), f"{what}: db off at {np.argwhere(bad)[0]}"


def problem(M, d_out, seed):
    return synth.gaussian_bf16((M, d_out), 1.0, seed), synth.gaussian_bf16((M, d_out), 2.5, seed + 1)


@pytest.mark.parametrize("act", oe.ACTS)
@pytest.mark.parametrize("M,d_out", [(1, 8), (3, 264), (17, 2056), (128, 2048), (129, 4104), (300, 8200), (1000, 136),
                                     (5000, 72), (40, 14336)])
def test_epilogue_backward(M, d_out, act):
    dY, Z = problem(M, d_out, M + d_out)
    dZ, db = slr.epilogue_backward(to_dev(dY), to_dev(Z), act, out=torch.empty((M, d_out), dtype=torch.bfloat16, device="cuda"))
    check(dZ, db, dY, Z, act, f"{M}x{d_out} {act}")


def test_wide_slopes_and_specials():
    """Every magnitude of Z from the smallest to the largest, its infinities and NaN."""
    z = torch.tensor([s * 2.0 ** e for e in range(-120, 121, 3) for s in (1.0, -1.0, 1.5, -1.5)], dtype=torch.bfloat16)
    z = torch.cat([z, torch.zeros(-len(z) % 8)]).to(torch.bfloat16).reshape(1, -1).cuda()
    one = torch.ones_like(z)
    for act in oe.ACTS:
        dZ, _ = slr.epilogue_backward(one, z, act, out=torch.empty_like(z))
        zz = np.clip(z.double().cpu().numpy(), -1e3, 1e3)   # the slopes are at their limits there
        assert np.abs(dZ.double().cpu().numpy() - oe.act_slope(zz, act)).max() <= 2.0 ** -8 * 1.13 + 2.0 ** -16
    inf = float("inf")
    z = torch.tensor([[inf, -inf, float("nan"), 0.0, 1.0, -1.0, 2.0, -2.0]], dtype=torch.bfloat16, device="cuda")
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        dZ, db = slr.epilogue_backward(torch.ones_like(z), z, act)
        assert dZ[0, 0] == 1.0 and dZ[0, 1] == 0.0 and torch.isfinite(dZ[0, 3:]).all()
        assert (dZ[0, 2] == 0.0) if act == "relu" else torch.isnan(dZ[0, 2])


def test_in_place_optional_outputs_and_empty_batch():
    dY, Z = problem(333, 520, 4)
    for into in ("dY", "Z"):
        g, z = to_dev(dY), to_dev(Z)
        dZ, db = slr.epilogue_backward(g, z, "gelu", out=g if into == "dY" else z)
        assert dZ.data_ptr() == (g if into == "dY" else z).data_ptr()
        check(dZ, db, dY, Z, "gelu", f"in place in {into}")
    dZ, none = slr.epilogue_backward(to_dev(dY), to_dev(Z), "silu", want_dbias=False)
    assert none is None
    check(dZ, None, dY, Z, "silu", "without db")
    g = to_dev(dY)
    same, db = slr.epilogue_backward(g, None, "none")
    assert same is g
    check(None, db, dY, Z, "none", "db alone")
    e = torch.empty((0, 520), dtype=torch.bfloat16, device="cuda")
    dZ, db = slr.epilogue_backward(e, e, "relu")
    assert dZ.shape == (0, 520) and torch.count_nonzero(db) == 0


def test_deterministic_and_captured():
    dY, Z = problem(700, 2048, 8)
    g, z = to_dev(dY), to_dev(Z)
    first = slr.epilogue_backward(g, z, "gelu_tanh")
    assert all(torch.equal(a, b) for a, b in zip(first, slr.epilogue_backward(g, z, "gelu_tanh")))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dZ, db = slr.epilogue_backward(g, z, "gelu_tanh")
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dZ, first[0]) and torch.equal(db, first[1])


def test_gradient_of_the_forward_by_differences():
    """<dY, Y(bias)> through slr.forward_epilogue: the column sums are its derivative along a bias step."""
    M, d_out, d_in = 64, 264, 256
    X = to_dev(synth.gaussian_bf16((M, d_in), 1.0, 1))
    vals, meta = slr.pack_2to4(to_dev(synth.gaussian_bf16((d_out, d_in), 0.05, 2)))
    dYb = synth.gaussian_bf16((M, d_out), 1.0, 3)
    Z = torch.empty((M, d_out), dtype=torch.bfloat16, device="cuda")
    for act in ("gelu", "gelu_tanh", "silu"):
        zero = torch.zeros(d_out, dtype=torch.bfloat16, device="cuda")
        slr.forward_epilogue(X, vals, meta, None, None, bias=zero, act=act, preact=Z)
        _, db = slr.epilogue_backward(to_dev(dYb), Z, act)
        step, dy = 0.125, bits_to_f64(dYb)
        ys = [bits_to_f64(from_dev(slr.forward_epilogue(X, vals, meta, None, None, bias=zero + s, act=act)))
              for s in (step, -step)]
        num = (dy * (ys[0] - ys[1])).sum(0) / (2 * step)
        # The quotient's own error: step^2 / 6 of the third derivative (below 2 for
        # these activations), and 2^-8 |Y| of rounding at each end; Z's rounding moves
        # the slope by at most 2^-8 |Z| (second derivative below 1).
        tol = (np.abs(dy) * (step ** 2 / 3 + 2.0 ** -8 * (np.abs(ys[0]) + np.abs(ys[1])) / (2 * step)
                             + 2.0 ** -8 * np.abs(bits_to_f64(from_dev(Z))))).sum(0)
        assert np.all(np.abs(db.cpu().numpy() - num) <= tol), act
