"""The fine-tuning operators as a training step uses them: a small compressed
network (an MLP block with bias, GELU and residual, then a head) distilled from a
teacher's top logits, its gradients carried down through every operator, against
the same network in fp64 by automatic differentiation.

Tolerance: the step rounds at most 14 tensors to bf16 between the input and any
gradient (two pre-activations and outputs, T and G of three layers, logits,
dlogits, three dX, two dZ), each within 2^-8 relative of its own norm (half a
step), in terms that the following products pass on without cancellation beyond
their norm: 14 x 2^-8 = 0.055 of the gradient's Frobenius norm."""
import numpy as np
import pytest
import torch

import oracle.epilogue as oe
import synth
from gpu_util import bits_to_f64, to_dev

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_rank_linear_02_b200 as slr

M, D, F, N, K, R = 200, 256, 512, 1000, 16, 16


def layer(d_out, d_in, seed):
    vals, meta = slr.pack_2to4(to_dev(synth.gaussian_bf16((d_out, d_in), d_in ** -0.5, seed)))
    return {"vals": vals, "meta": meta, "U": to_dev(synth.gaussian_bf16((d_out, R), 0.1, seed + 1)),
            "V": to_dev(synth.gaussian_bf16((R, d_in), d_in ** -0.5, seed + 2)),
            "bias": to_dev(synth.gaussian_bf16((d_out,), 0.1, seed + 3))}


def network():
    up, down, head = layer(F, D, 10), layer(D, F, 20), layer(N, D, 30)
    X = to_dev(synth.gaussian_bf16((M, D), 1.0, 1))
    g = np.random.default_rng(2)
    idx = np.stack([g.choice(N, size=K, replace=False) for _ in range(M)]).astype(np.int32)
    teacher = (g.standard_normal((M, K)) * 2).astype(np.float32)
    idx[M - 9:] = -1                                       # padded tokens
    w = np.full(M, 1.0 / (M - 9), np.float32)
    w[M - 9:] = 0
    return up, down, head, X, torch.from_numpy(idx).cuda(), torch.from_numpy(teacher).cuda(), torch.from_numpy(w).cuda()


def step(up, down, head, X, idx, teacher, w):
    """Loss per token and the gradients, all by this library."""
    f = lambda p: (p["vals"], p["meta"], p["U"], p["V"])  # noqa: E731
    Z = torch.empty((M, F), dtype=torch.bfloat16, device="cuda")
    A = slr.forward_epilogue(X, *f(up), bias=up["bias"], act="gelu", preact=Z)
    H = slr.forward_epilogue(A, *f(down), bias=down["bias"], residual=X)
    logits = slr.forward_epilogue(H, *f(head), bias=head["bias"])
    loss, dlogits = slr.distill_loss_grad(logits, idx, teacher, w, tau=2.0, out=logits)   # in place
    _, db3 = slr.epilogue_backward(dlogits, None, "none")
    dU3, dV3 = slr.lora_backward(H, dlogits, head["U"], head["V"])
    dH = slr.input_backward(dlogits, *f(head))
    _, db2 = slr.epilogue_backward(dH, None, "none")
    dU2, dV2 = slr.lora_backward(A, dH, down["U"], down["V"])
    dA = slr.input_backward(dH, *f(down))
    dZ, db1 = slr.epilogue_backward(dA, Z, "gelu", out=dA)
    dU1, dV1 = slr.lora_backward(X, dZ, up["U"], up["V"])
    dX = slr.input_backward(dZ, *f(up))
    return loss, {"U1": dU1, "V1": dV1, "b1": db1, "U2": dU2, "V2": dV2, "b2": db2, "U3": dU3, "V3": dV3, "b3": db3,
                  "X through the block": dX, "X through the residual": dH}


def reference(up, down, head, X, idx, teacher, w):
    """The same by automatic differentiation in fp64."""
    p = {}
    for n, q in (("1", up), ("2", down), ("3", head)):
        S = oe.dense(q["vals"].view(torch.int16).cpu().numpy().view(np.uint16), q["meta"].cpu().numpy())
        p["S" + n] = torch.from_numpy(S).cuda()
        for a in ("U", "V"):
            p[a + n] = q[a].double().requires_grad_()
        p["b" + n] = q["bias"].double().requires_grad_()
    lin = lambda x, n: x @ p["S" + n].T + (x @ p["V" + n].T) @ p["U" + n].T + p["b" + n]  # noqa: E731
    X1, X2 = X.double().requires_grad_(), X.double().requires_grad_()   # the block's input, the residual's
    h = lin(torch.nn.functional.gelu(lin(X1, "1")), "2") + X2
    logq = torch.log_softmax(lin(h, "3") / 2.0, dim=1)
    live = (idx >= 0).all(dim=1)
    logp = torch.log_softmax(teacher.double() / 2.0, dim=1)
    loss = 4.0 * (logp.exp() * (logp - logq.gather(1, idx.clamp(min=0).long()))).sum(1) * live
    (loss * w.double()).sum().backward()
    grads = {k: p[k].grad for k in ("U1", "V1", "b1", "U2", "V2", "b2", "U3", "V3", "b3")}
    return loss.detach(), {**grads, "X through the block": X1.grad, "X through the residual": X2.grad}


def compare(got, want):
    loss, grads = got
    wl, wg = want
    assert float((loss.double() - wl).norm() / wl.norm()) <= 4 * 2.0 ** -8     # four roundings before the loss
    for k, g in grads.items():
        rel = float((g.double() - wg[k]).norm() / wg[k].norm())
        assert rel <= 14 * 2.0 ** -8, f"{k}: {rel}"


def test_training_step_gradients():
    net = network()
    got = step(*net)
    torch.cuda.synchronize()
    slr.check_kernel_error()
    compare(got, reference(*net))
    pad = got[1]["X through the residual"][M - 9:]
    assert torch.count_nonzero(pad) == 0 and torch.count_nonzero(got[0][M - 9:]) == 0


def test_training_step_captured():
    """The whole step as one CUDA graph, replayed on changed parameters, beside eager calls."""
    net = network()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*net)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(*net)
    g.replay()
    torch.cuda.synchronize()
    eager = step(*net)
    torch.cuda.synchronize()
    assert torch.equal(got[0], eager[0]) and all(torch.equal(got[1][k], eager[1][k]) for k in eager[1])
    net[0]["U"].mul_(0.5)
    net[1]["bias"].add_(0.25)
    g.replay()
    torch.cuda.synchronize()
    slr.check_kernel_error()
    compare(got, reference(*net))


def test_single_token_decode_of_the_network():
    """One token through the block, as serving calls it: the bits of the batch's row up to its own rounding."""
    up, down, head, X, *_ = network()
    f = lambda p: (p["vals"], p["meta"], p["U"], p["V"])  # noqa: E731
    x = X[:1].contiguous()
    A = slr.forward_epilogue(x, *f(up), bias=up["bias"], act="gelu")
    H = x.clone()
    slr.forward_epilogue(A, *f(down), bias=down["bias"], residual=H, out=H)
    S = [torch.from_numpy(oe.dense(q["vals"].view(torch.int16).cpu().numpy().view(np.uint16), q["meta"].cpu().numpy())).cuda()
         for q in (up, down)]
    lin = lambda x, s, q: x @ s.T + (x @ q["V"].double().T) @ q["U"].double().T + q["bias"].double()  # noqa: E731
    want = lin(torch.nn.functional.gelu(lin(x.double(), S[0], up)), S[1], down) + x.double()
    assert float((H.double() - want).norm() / want.norm()) <= 3 * 2.0 ** -8
