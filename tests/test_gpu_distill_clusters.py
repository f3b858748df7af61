"""The distillation loss where clusters share a row, with its CTAs started at
odd times: beside other grids that hold part of the GPU.  The same bits as alone."""
import pytest
import torch

from test_gpu_distill import all_three, problem

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_rank_linear_02_b200 as slr


@pytest.mark.parametrize("M,n", [(1, 131072), (1, 16400), (3, 20000), (40, 33000), (90, 20001), (700, 66000), (160, 300000)])
def test_clusters_beside_other_grids(M, n):
    z, idx, t, w = (x.cuda() for x in problem(M, n, 24, M + n))
    fwd, step = slr.distill_forward(z, idx, t), slr.distill_loss_grad(z, idx, t, w)
    a = torch.randn((2048, 2048), device="cuda").bfloat16()
    x = torch.randn(1 << 22, device="cuda")
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []
    with torch.cuda.stream(side):
        for _ in range(40):
            a @ a
            x.sin()
    for _ in range(20):
        got.append((slr.distill_forward(z, idx, t), slr.distill_loss_grad(z, idx, t, w)))
    torch.cuda.synchronize()
    for f, s in got:
        assert all(torch.equal(p, q) for p, q in zip(f, fwd)) and all(torch.equal(p, q) for p, q in zip(s, step))


@pytest.mark.parametrize("M,n", [(1, 16392), (7, 50001), (2, 70000), (1, 262147)])
@pytest.mark.parametrize("k", [1, 40])
def test_clusters_against_the_definition(M, n, k):
    all_three(*problem(M, n, k, M * n + k), 1.5, f"{M}x{n} k={k}")
