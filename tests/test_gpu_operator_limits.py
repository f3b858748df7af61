"""GPU tests of what the fine-tuning operators' descriptions allow at the edges:
elements past 2^31, infinite pre-activations, rows without a finite logit, calls
on two streams at once, one workspace in two captured graphs.  Parity checks and
their tolerances are those of each operator's own tests."""
import pytest
import torch

import oracle.epilogue as oe
import test_gpu_epilogue as te
import test_gpu_epilogue_backward as tb
import test_gpu_input_backward as ti
from gpu_util import to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_rank_linear_02_b200 as slr

FAR, WIDE, LAST = 262200, 8192, 37   # the last rows start past element 2^31 of a FAR x WIDE matrix


def far(rows: torch.Tensor) -> torch.Tensor:
    big = torch.zeros((FAR, rows.shape[1]), dtype=rows.dtype, device="cuda")
    big[FAR - LAST:] = rows
    return big


def test_forward_past_32_bits():
    assert (FAR - LAST) * WIDE > 2 ** 31
    L = te.Layer(LAST, WIDE, 128, 8, 3)
    X, vals, meta, U, V = L.device()
    Z = torch.empty((FAR, WIDE), dtype=torch.bfloat16, device="cuda")
    Y = slr.forward_epilogue(far(X), vals, meta, U, V, bias=to_dev(L.bias), act="silu", residual=far(to_dev(L.R)), preact=Z)
    slr.check_kernel_error()
    te.check(Y[FAR - LAST:], Z[FAR - LAST:], L, "silu", True, True, "far rows")


def test_epilogue_backward_past_32_bits():
    dY, Z = tb.problem(LAST, WIDE, 4)
    dZ, db = slr.epilogue_backward(far(to_dev(dY)), far(to_dev(Z)), "gelu")
    tb.check(dZ[FAR - LAST:], db, dY, Z, "gelu", "far rows")   # the zero rows add nothing to db
    assert torch.count_nonzero(dZ[: FAR - LAST]) == 0


def test_input_backward_past_32_bits():
    p = ti.Problem(LAST, 8, WIDE, 8, 5)
    dY, *layer = p.device()
    dX = slr.input_backward(far(dY), *layer)
    slr.check_kernel_error()
    p.check(dX[FAR - LAST:], "far rows")
    assert torch.count_nonzero(dX[: FAR - LAST]) == 0


@pytest.mark.parametrize("M,path", [(1, "decode"), (6, "tensor"), (100, "tensor")])
@pytest.mark.parametrize("act", oe.ACTS)
def test_infinite_pre_activation(M, path, act):
    L = te.Layer(M, 264, 256, 8, 5)
    ops, bias = L.device(), to_dev(L.bias)
    clean = slr.forward_epilogue(*ops, bias=bias, act=act, path=path)
    bias[5] = float("-inf")
    Z = torch.empty_like(clean)
    Y = slr.forward_epilogue(*ops, bias=bias, act=act, preact=Z, path=path)
    assert (Z[:, 5] == float("-inf")).all()
    if act == "none":
        assert (Y[:, 5] == float("-inf")).all()
    elif act == "relu":
        assert (Y[:, 5] == 0).all()
    else:
        assert torch.isnan(Y[:, 5]).all()
    others = [c for c in range(264) if c != 5]
    assert torch.equal(Y[:, others], clean[:, others])


def test_row_without_a_finite_logit():
    z = torch.randn((3, 5000), device="cuda").bfloat16()
    z[1] = float("-inf")
    idx = torch.arange(4, dtype=torch.int32, device="cuda").repeat(3, 1)
    t, w = torch.zeros((3, 4), device="cuda"), torch.ones(3, device="cuda")
    loss, lse = slr.distill_forward(z, idx, t)
    loss2, dz = slr.distill_loss_grad(z, idx, t, w)
    dz2 = slr.distill_backward(z, idx, t, lse, w)
    for a in (loss, loss2, dz, dz2):
        assert torch.isnan(a[1]).all() and torch.isfinite(a[[0, 2]]).all()


def calls():
    """One call of each operator, on operands of its own: name -> (function, its result)."""
    L = te.Layer(300, 1032, 512, 64, 7)
    ops, R = L.device(), to_dev(L.R)
    p = ti.Problem(64, 4096, 512, 64, 8)
    small = te.Layer(20, 1032, 512, 64, 9)
    sops = small.device()
    dY, Z = (to_dev(b) for b in tb.problem(300, 1032, 10))
    z = torch.randn((64, 20001), device="cuda").bfloat16()
    idx = torch.randint(0, 20001, (64, 16), dtype=torch.int32, device="cuda")
    t, w = torch.randn((64, 16), device="cuda"), torch.rand(64, device="cuda")
    pops = p.device()
    return [lambda: slr.forward_epilogue(*ops, act="gelu", residual=R), lambda: slr.forward_epilogue(*sops, act="silu"),
            lambda: slr.input_backward(*pops), lambda: slr.epilogue_backward(dY, Z, "gelu_tanh"),
            lambda: slr.distill_loss_grad(z, idx, t, w)]


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_streams_at_once():
    fs = calls()
    want = [f() for f in fs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for turn in range(4):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                for i in range(len(fs)):
                    j = (i + 2 * n + turn) % len(fs)
                    got[n].append((j, fs[j]()))
    torch.cuda.synchronize()
    slr.check_kernel_error()
    assert all(same(r, want[j]) for g in got for j, r in g)


def test_one_workspace_in_two_graphs():
    p, q = ti.Problem(64, 4096, 512, 64, 11), ti.Problem(64, 4096, 512, 64, 12)
    ws = torch.empty(slr.input_backward_workspace_size(64, 4096, 512, 64), dtype=torch.uint8, device="cuda")
    L = te.Layer(300, 1032, 512, 64, 13)
    lops = L.device()
    lws = torch.empty(slr.workspace_size(300, 1032, 512, 64), dtype=torch.uint8, device="cuda")
    graphs, outs, want = [], [], []
    for ops, act in ((p.device(), "gelu"), (q.device(), "relu")):
        want.append((slr.input_backward(*ops), slr.forward_epilogue(*lops, act=act)))
        outs.append(tuple(torch.empty_like(x) for x in want[-1]))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            slr.input_backward(*ops, out=outs[-1][0], workspace=ws)
            slr.forward_epilogue(*lops, act=act, out=outs[-1][1], workspace=lws)
        graphs.append((g, ops))
    for _ in range(3):
        for g, _ops in graphs:
            g.replay()
    torch.cuda.synchronize()
    slr.check_kernel_error()
    assert all(same(a, b) for a, b in zip(outs, want))
