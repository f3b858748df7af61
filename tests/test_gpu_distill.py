"""GPU parity of the distillation operators (slr_distill_forward / _backward /
_loss_grad) against the fp64 definition (oracle/distill.py).

Tolerances, from the arithmetic, with R the largest |z| / tau or |t| / tau of the
token: an exponent or logarithm's argument is rounded a few times at 2^-24 of at
most 2 R, the approximate 2^x is within 2^-22, partial sums join in at most 16
steps (2^-22 each) after chains of at most 64 x ceil(n / 32768) additions.  So
log q is within E = 2^-17 + 2^-21 R (n <= 300000), p and q within E relative;
dlogits is rounded to bf16 once (2^-8 relative)."""
import numpy as np
import pytest
import torch

import oracle.distill as od

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_rank_linear_02_b200 as slr


def problem(M, n, k, seed, std=2.5):
    g = np.random.default_rng(seed)
    z = torch.from_numpy(g.standard_normal((M, n)).astype(np.float32) * std).bfloat16()
    idx = np.stack([g.choice(n, size=min(k, n), replace=False) for _ in range(M)]).astype(np.int32)
    if k > n:
        idx = np.concatenate([idx, np.full((M, k - n), -1, np.int32)], axis=1)
    t = (g.standard_normal((M, k)) * 2).astype(np.float32)
    w = (g.random(M) + 0.5).astype(np.float32)
    return z, torch.from_numpy(idx), torch.from_numpy(t), torch.from_numpy(w)


def tolerances(z, idx, t, w, tau):
    zf, tf = z.double().numpy(), t.double().numpy()
    with np.errstate(invalid="ignore", over="ignore"):
        loss, lse, dz, spread = od.distill(zf, idx.numpy(), tf, tau)
    big = lambda x: np.abs(np.where(np.abs(x) < 1e30, x, 0)).max(1)  # noqa: E731  (past that: masks, whose p or q is 0)
    R = np.maximum(big(zf), big(tf)) / tau
    E = 2.0 ** -17 + 2.0 ** -21 * R
    return loss, lse, dz, tau ** 2 * E * (1 + spread) + 1e-6 * tau ** 2 * spread, E


def check_loss(loss, z, idx, t, w, tau, what, lse=None):
    want, wl, _, tol, E = tolerances(z, idx, t, w, tau)
    got = loss.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), f"{what}: loss {got[np.abs(got - want) > tol][:3]} vs {want[np.abs(got - want) > tol][:3]}"
    if lse is not None:
        assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= E + 2.0 ** -23 * np.abs(wl)), f"{what}: lse"


def check_grad(dz, z, idx, t, w, tau, what):
    _, _, want, _, E = tolerances(z, idx, t, w, tau)
    wd = w.double().numpy()[:, None]
    want = want * wd
    p = np.zeros(want.shape)   # what is subtracted, for its share of the error
    for m in range(want.shape[0]):
        there = [(i, x) for i, x in zip(idx[m].tolist(), t[m].tolist()) if 0 <= i < want.shape[1] and x != -np.inf]
        if there:
            x = np.array([x for _, x in there]) / tau
            e = np.exp(x - x.max())
            np.add.at(p[m], [i for i, _ in there], e / e.sum())
    err = 2 * E[:, None] * (np.abs(want) + 2 * tau * np.abs(wd) * p)
    tol = err + 2.0 ** -8 * (np.abs(want) + err) + 1e-37
    got = dz.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: dz off at {np.argwhere(bad)[0]}: {got[bad][0]} vs {want[bad][0]} ({bad.sum()})"


def all_three(z, idx, t, w, tau, what):
    zd, i, td, wd = z.cuda(), idx.cuda(), t.cuda(), w.cuda()
    loss, lse = slr.distill_forward(zd, i, td, tau=tau)
    check_loss(loss, z, idx, t, w, tau, what, lse)
    dz = slr.distill_backward(zd, i, td, lse, wd, tau=tau)
    check_grad(dz, z, idx, t, w, tau, what + " backward")
    loss2, dz2 = slr.distill_loss_grad(zd, i, td, wd, tau=tau)
    check_loss(loss2, z, idx, t, w, tau, what + " step")   # its sums may be cut elsewhere: not the same bits
    check_grad(dz2, z, idx, t, w, tau, what + " step")


@pytest.mark.parametrize("M,n,k", [(1, 1, 1), (3, 7, 2), (2, 8, 8), (5, 100, 64), (4, 1023, 20), (3, 8192, 256),
                                   (3, 8200, 3), (2, 32000, 64), (3, 50001, 20), (2, 131072, 64), (1, 131071, 1000),
                                   (2, 300000, 8), (400, 4099, 5)])
@pytest.mark.parametrize("tau", [1.0, 3.0])
def test_distill_shapes(M, n, k, tau):
    all_three(*problem(M, n, k, M + n + k), tau, f"{M}x{n} k={k} tau={tau}")


@pytest.mark.parametrize("k", [1, 31, 128, 129, 1024])
@pytest.mark.parametrize("tau", [0.25, 10.0])
def test_list_lengths_and_temperatures(k, tau):
    all_three(*problem(6, 2000, k, k), tau, f"k={k} tau={tau}")


def test_absent_duplicate_and_masked_entries():
    M, n, k = 9, 5003, 12
    z, idx, t, w = problem(M, n, k, 3)
    idx[0] = -1                                  # nothing listed
    idx[1, 3:] = -7                              # a short list
    idx[2, 4], idx[2, 5] = n, 2 ** 31 - 1        # columns past the vocabulary
    idx[3, 1] = idx[3, 0]                        # listed twice
    idx[4, :] = idx[4, 0]                        # listed k times
    t[5] = -np.inf                               # no mass
    t[6, :6] = -np.inf
    t[7, 2] = -3.4e38                            # the type's lowest value
    all_three(z, idx, t, w, 1.0, "masks")
    all_three(z, idx, t, w, 2.0, "masks, tau 2")
    loss, lse = slr.distill_forward(z.cuda(), idx.cuda(), t.cuda())
    assert loss[0] == 0 and lse[0] == 0 and loss[5] == 0 and lse[5] == 0


def test_rows_without_entries_or_weight_ignore_their_logits():
    M, n, k = 6, 4100, 4
    z, idx, t, w = problem(M, n, k, 5)
    z[1] = float("nan")
    z[2, 17] = float("inf")
    idx[1] = -1
    w[2] = 0.0
    zd, i, td, wd = z.cuda(), idx.cuda(), t.cuda(), w.cuda()
    loss, lse = slr.distill_forward(zd, i, td)
    assert loss[1] == 0 and torch.isnan(loss[2])
    dz = slr.distill_backward(zd, i, td, lse, wd)
    _, dz2 = slr.distill_loss_grad(zd, i, td, wd)
    for d in (dz, dz2):
        assert torch.count_nonzero(d[1]) == 0 and torch.count_nonzero(d[2]) == 0
        assert torch.isfinite(d[[0, 3, 4, 5]]).all()
    z2, keep = z.clone(), [0, 3, 4, 5]
    check_grad(dz[keep], z2[keep], idx[keep], t[keep], w[keep], 1.0, "beside masked rows")


def test_masked_vocabulary_and_nan():
    M, n, k = 4, 3001, 5
    z, idx, t, w = problem(M, n, k, 8)
    z[:, 100:2000] = float("-inf")               # columns that may not be sampled
    idx[:] = torch.arange(k) + 2500
    all_three(z, idx, t, w, 1.0, "-inf columns")
    low = torch.finfo(torch.bfloat16).min        # the type's lowest value as the mask
    zl = z.clone()
    zl[:, 100:2000] = low
    zl[0, :2400] = low
    all_three(zl, idx, t, w, 1.0, "lowest-value columns")
    all_three(zl, idx, t, w, 0.5, "lowest-value columns, tau 0.5")
    zl[3] = low                                  # every column masked: q is uniform
    loss, dz = slr.distill_loss_grad(zl.cuda(), idx.cuda(), t.cuda(), w.cuda())
    check_loss(loss, zl, idx, t, w, 1.0, "all lowest")
    check_grad(dz, zl, idx, t, w, 1.0, "all lowest")
    idx[1, 0] = 150                              # a listed column with q = 0
    loss, lse = slr.distill_forward(z.cuda(), idx.cuda(), t.cuda())
    assert loss[1] == float("inf") and torch.isfinite(loss[[0, 2, 3]]).all()
    dz = slr.distill_backward(z.cuda(), idx.cuda(), t.cuda(), lse, w.cuda())
    check_grad(dz, z, idx, t, w, 1.0, "q = 0 at a listed column")
    z[2, 5] = float("nan")
    t[3, 1] = float("nan")
    loss, dz = slr.distill_loss_grad(z.cuda(), idx.cuda(), t.cuda(), w.cuda())
    assert torch.isnan(loss[2]) and torch.isnan(loss[3]) and torch.isfinite(loss[0])
    assert torch.isnan(dz[2]).any() and torch.isnan(dz[3]).any() and torch.isfinite(dz[0]).all()


@pytest.mark.parametrize("off_in,off_out", [(0, 0), (1, 1), (3, 3), (0, 1), (5, 2)])
def test_padded_rows_alignments_and_what_lies_behind(off_in, off_out):
    M, n, k, ld = 7, 2077, 9, 2100
    z, idx, t, w = problem(M, n, k, off_in * 10 + off_out)
    big = torch.full((M, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[:, off_in:off_in + n] = z.cuda()
    out = torch.full((M + 1, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out[:M, off_out:off_out + n]
    loss, got = slr.distill_loss_grad(big[:, off_in:off_in + n], idx.cuda(), t.cuda(), w.cuda(), out=view)
    check_loss(loss, z, idx, t, w, 1.0, "padded")
    check_grad(got, z, idx, t, w, 1.0, "padded")
    mask = torch.ones_like(out, dtype=torch.bool)
    mask[:M, off_out:off_out + n] = False
    assert torch.all(out[mask] == 7.0), "columns or rows behind the problem were written"


@pytest.mark.parametrize("M,n", [(5, 1000), (3, 50001), (2, 131072), (1, 290001)])
def test_in_place(M, n):
    z, idx, t, w = problem(M, n, 16, n)
    i, td, wd = idx.cuda(), t.cuda(), w.cuda()
    loss, dz = slr.distill_loss_grad(z.cuda(), i, td, wd)
    zin = z.cuda()
    loss2, dz2 = slr.distill_loss_grad(zin, i, td, wd, out=zin)
    assert dz2.data_ptr() == zin.data_ptr() and torch.equal(dz, dz2) and torch.equal(loss, loss2)
    zin = z.cuda()
    _, lse = slr.distill_forward(zin, i, td)
    ref = slr.distill_backward(zin, i, td, lse, wd)
    got = slr.distill_backward(zin, i, td, lse, wd, out=zin)
    assert torch.equal(ref, got)


def test_gradient_by_differences():
    """Central differences of the fp64 definition at the kernel's own inputs, column by column."""
    z, idx, t, w = problem(1, 40, 6, 2)
    dz = slr.distill_loss_grad(z.cuda(), idx.cuda(), t.cuda(), torch.ones(1).cuda(), tau=2.0)[1].double().cpu().numpy()
    zf, h = z.double().numpy(), 1e-5
    for v in range(40):
        e = np.zeros_like(zf)
        e[0, v] = h
        num = (od.distill(zf + e, idx.numpy(), t.double().numpy(), 2.0)[0] -
               od.distill(zf - e, idx.numpy(), t.double().numpy(), 2.0)[0])[0] / (2 * h)
        assert abs(dz[0, v] - num) <= 2.0 ** -8 * abs(num) + 1e-6


def test_deterministic_captured_and_second_stream():
    z, idx, t, w = problem(64, 50001, 32, 1)
    zd, i, td, wd = z.cuda(), idx.cuda(), t.cuda(), w.cuda()
    first = slr.distill_loss_grad(zd, i, td, wd)
    assert all(torch.equal(a, b) for a, b in zip(first, slr.distill_loss_grad(zd, i, td, wd)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = slr.distill_loss_grad(zd, i, td, wd)
    g.replay()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    with torch.cuda.stream(s):
        other = slr.distill_loss_grad(zd, i, td, wd)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    none = slr.distill_forward(zd[:0], i[:0], td[:0])
    assert none[0].shape == (0,)


def test_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31: the last of 16500 padded rows of 131100."""
    M, n, ld, k = 16500, 131072, 131100, 4
    big = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")
    big.fill_(0)
    z, idx, t, w = problem(2, n, k, 6)
    big[M - 2:, :n] = z.cuda()
    i = torch.full((M, k), -1, dtype=torch.int32, device="cuda")
    i[M - 2:] = idx.cuda()
    td, wd = torch.zeros((M, k), device="cuda"), torch.zeros(M, device="cuda")
    td[M - 2:], wd[M - 2:] = t.cuda(), w.cuda()
    loss, dz = slr.distill_loss_grad(big[:, :n], i, td, wd, out=big[:, :n])
    check_loss(loss[M - 2:], z, idx, t, w, 1.0, "far rows")
    check_grad(dz[M - 2:], z, idx, t, w, 1.0, "far rows")
    assert torch.count_nonzero(loss[:M - 2]) == 0
