"""Distillation's gradients at temperatures and logits so large in units of tau
that an fp32 lse no longer holds them (|lse| > 64).

Tolerances: an exponent's argument (z - max) / tau is a difference (2^-24 relative)
times a factor of two roundings, minus a logarithm: within 2^-21 of its size, and
where it is below -128 its q is under 2^-126.  The approximate 2^x and the sums are
within 2^-17 (as in test_gpu_distill.py).  So q and p are within E = 2^-17 +
2^-21 x 128 relative, whatever |z| / tau is; dlogits is rounded to bf16 once."""
import numpy as np
import pytest
import torch

import oracle.distill as od

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_rank_linear_02_b200 as slr

E = 2.0 ** -17 + 2.0 ** -21 * 128


def near_teacher(M, n, k, seed, std):
    """Logits, and a teacher that lists their k largest as they are: p is close to q."""
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn((M, n), generator=g) * std).bfloat16()
    top = z.float().topk(k, dim=1)
    w = torch.rand(M, generator=g) + 0.5
    return z, top.indices.to(torch.int32), top.values.contiguous(), w


def check(dz, z, idx, t, w, tau, what):
    z, idx, t, w = (x.double().cpu().numpy() for x in (z, idx, t, w))
    _, _, want, _ = od.distill(z, idx.astype(np.int64), t, tau)
    want *= w[:, None]
    x = (t - t.max(1, keepdims=True)) / tau
    e = np.exp(x)
    p = np.zeros_like(want)
    for m in range(z.shape[0]):
        np.add.at(p[m], idx[m].astype(np.int64), e[m] / e[m].sum())
    err = 2 * E * (np.abs(want) + 2 * tau * w[:, None] * p)
    tol = err + 2.0 ** -8 * (np.abs(want) + err) + 1e-37
    got = dz.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: dz off at {np.argwhere(bad)[0]}: {got[bad][0]} vs {want[bad][0]} ({bad.sum()})"


@pytest.mark.parametrize("M,n,k,std", [(3, 40, 4, 10.0), (4, 5000, 8, 10.0), (2, 20001, 16, 3.0), (1, 131072, 64, 5.0),
                                       (300, 9001, 8, 30.0)])
@pytest.mark.parametrize("tau", [1e-1, 1e-2, 1e-3, 1e-4])
def test_backward_where_lse_is_large(M, n, k, std, tau):
    args = near_teacher(M, n, k, n, std)
    z, idx, t, w = (x.cuda() for x in args)
    _, lse = slr.distill_forward(z, idx, t, tau=tau)
    dz = slr.distill_backward(z, idx, t, lse, w, tau=tau)
    _, step = slr.distill_loss_grad(z, idx, t, w, tau=tau)
    check(step, *args, tau, "loss_grad")
    check(dz, *args, tau, "backward")
    far = lse.abs() > 64
    assert (std / tau < 100 or far.any()) and torch.equal(dz[far], step[far])
    inplace = slr.distill_backward(z, idx, t, lse, w, tau=tau, out=z)
    assert torch.equal(inplace, dz)


@pytest.mark.parametrize("shift", [-80.0, -66.0, -60.0, 0.0, 50.0, 58.0, 70.0])
@pytest.mark.parametrize("n", [3001, 20001])
def test_rows_on_both_sides_of_the_border(n, shift):
    """Rows around |lse| = 64, next to ordinary ones and ones without weight or entries."""
    z, idx, t, w = near_teacher(6, n, 8, n, 1.0)
    z[:3] = (z[:3].float() + shift).bfloat16()
    t = z.float().gather(1, idx.long())
    w[1], idx[2] = 0.0, -1
    args = z, idx, t, w
    z, idx, t, w = (x.cuda() for x in args)
    _, lse = slr.distill_forward(z, idx, t)
    dz = slr.distill_backward(z, idx, t, lse, w)
    keep = [0, 3, 4, 5]
    check(dz[keep], *(x[keep] for x in args), 1.0, f"shift {shift}")
    assert torch.count_nonzero(dz[1:3]) == 0


def test_lse_that_overflows():
    """Logits whose z / tau is past fp32: the gradient is still the softmax's."""
    z, idx, t, w = near_teacher(3, 20001, 4, 7, 1.0)
    z[0, 17], z[1] = 3e38, torch.finfo(torch.bfloat16).min
    z[1, 5:9] = 3e38
    z, idx, t, w = (x.cuda() for x in (z, idx, t, w))
    idx[:2], t[:2] = 100, 0.0
    _, lse = slr.distill_forward(z, idx, t, tau=0.25)
    assert torch.isinf(lse[:2]).all()
    dz = slr.distill_backward(z, idx, t, lse, w, tau=0.25)
    want = torch.zeros((2, 20001), device="cuda")
    want[0, 17], want[1, 5:9] = 1.0, 0.25
    want[:, 100] = -1.0
    want = want * 0.25 * w[:2, None]
    err = (dz[:2].float() - want).abs()
    assert (err <= (E + 2.0 ** -8) * want.abs()).all()
    assert torch.equal(dz, slr.distill_loss_grad(z, idx, t, w, tau=0.25)[1])
