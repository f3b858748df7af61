"""Timing cases of the fine-tuning operators of the 2:4-sparse + low-rank layer.

Four operators, each with its cases, its plain form in elementary torch
operations and its definition in 64 bits:

* ``forward``  -- Y = act(X S^T + (X V^T) U^T + b) + R, the layer with bias,
  activation and residual in its epilogue (optionally the pre-activation Z);
* ``act_grad`` -- dZ = dY * act'(Z) and db = the column sums of dZ;
* ``dx``       -- dX = dY S + (dY U) V, the gradient of the layer's input;
* ``distill``  -- the loss tau^2 KL(p || q) of a student's logits against a
  teacher's top logits, and its gradient.

``own`` selects the framework's kernels instead of the plain forms.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")

# The most multiply-adds of a drawn layer case, and the most logits of a drawn
# distillation case: those of the largest listed ones.
MAX_MADDS = 2048 * 14336 * 4096
MAX_LOGITS = 4096 * 131072


def listed():
    return [
        # One decoded token through an output projection that adds to the residual stream.
        {"name": "forward 1 token 4096x4096", "op": "forward", "M": 1, "d_out": 4096, "d_in": 4096, "r": 64,
         "bias": True, "act": "none", "residual": True, "preact": False},
        # A small decode batch through a gate projection.
        {"name": "forward 16 tokens 14336x4096", "op": "forward", "M": 16, "d_out": 14336, "d_in": 4096, "r": 64,
         "bias": True, "act": "silu", "residual": False, "preact": False},
        # The first linear of an MLP in training: the pre-activation is kept for the backward pass.
        {"name": "forward 2048 tokens 14336x4096", "op": "forward", "M": 2048, "d_out": 14336, "d_in": 4096, "r": 64,
         "bias": True, "act": "gelu_tanh", "residual": False, "preact": True},
        # The second linear of an MLP on a ragged batch, added to the residual stream.
        {"name": "forward 777 tokens 4096x14336", "op": "forward", "M": 777, "d_out": 4096, "d_in": 14336, "r": 128,
         "bias": True, "act": "none", "residual": True, "preact": False},
        # Gradient through the activation: a short sequence.
        {"name": "act_grad 17 tokens 4096", "op": "act_grad", "M": 17, "d_out": 4096, "act": "silu"},
        # Gradient through the activation: a training batch of the MLP's first linear.
        {"name": "act_grad 2048 tokens 14336", "op": "act_grad", "M": 2048, "d_out": 14336, "act": "gelu_tanh"},
        # Input gradient of a square projection for a short sequence.
        {"name": "dx 64 tokens 4096x4096", "op": "dx", "M": 64, "d_out": 4096, "d_in": 4096, "r": 64},
        # Input gradient of the MLP's first linear for a training batch.
        {"name": "dx 2048 tokens 14336x4096", "op": "dx", "M": 2048, "d_out": 14336, "d_in": 4096, "r": 64},
        # Input gradient of the MLP's second linear on a ragged batch.
        {"name": "dx 777 tokens 4096x14336", "op": "dx", "M": 777, "d_out": 4096, "d_in": 14336, "r": 128},
        # Scoring one token against a teacher's stored top logits.
        {"name": "distill score 1 token 131072", "op": "distill", "pass": "forward", "M": 1, "n_vocab": 131072,
         "k": 64, "tau": 1.0, "pad": 0},
        # The backward pass on an odd vocabulary, whose rows start at any alignment, with padded tokens.
        {"name": "distill backward 1000 tokens 50001", "op": "distill", "pass": "backward", "M": 1000,
         "n_vocab": 50001, "k": 20, "tau": 2.0, "pad": 37},
        # Loss and gradient of a training batch.
        {"name": "distill step 4096 tokens 131072", "op": "distill", "pass": "step", "M": 4096, "n_vocab": 131072,
         "k": 64, "tau": 1.0, "pad": 100},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["forward", "act_grad", "dx", "distill"])
    if op == "distill":
        n = spread(100, 131072)
        m = spread(1, min(4096, MAX_LOGITS // n))
        return {"op": op, "pass": rng.choice(["forward", "backward", "step"]), "M": m, "n_vocab": n,
                "k": spread(1, min(256, n)), "tau": rng.choice([0.5, 1.0, 2.0, 4.0]), "pad": rng.randint(0, m // 8)}
    if op == "act_grad":
        return {"op": op, "M": spread(1, 2048), "d_out": 8 * spread(1, 1792), "act": rng.choice(ACTS[1:])}
    d_out, d_in = 8 * spread(4, 1792), 128 * spread(1, 112)
    m = spread(1, min(2048, MAX_MADDS // (d_out * d_in)))
    r = 8 * spread(1, 32)
    if op == "dx":
        return {"op": op, "M": m, "d_out": d_out, "d_in": d_in, "r": r}
    return {"op": op, "M": m, "d_out": d_out, "d_in": d_in, "r": rng.choice([0, r, r]), "bias": rng.random() < 0.7,
            "act": rng.choice(ACTS), "residual": rng.random() < 0.5, "preact": rng.random() < 0.4}


# ---------------------------------------------------------------- inputs
def _pack(w):
    """The two largest magnitudes of every four columns: (values, index nibbles, two groups a byte)."""
    rows, cols = w.shape
    four = w.view(rows, cols // 4, 4)
    a = list(four.abs().unbind(2))
    # Position i stays when fewer than two of the others beat it (the lower index wins a tie).
    beaten = [sum((a[j] >= a[i] if j < i else a[j] > a[i]).to(torch.uint8) for j in range(4) if j != i) for i in range(4)]
    stays = [b < 2 for b in beaten]
    one, two, three = (torch.full_like(beaten[0], i) for i in (1, 2, 3))
    first = torch.where(stays[0], 0, torch.where(stays[1], one, two))
    second = torch.where(stays[3], three, torch.where(stays[2], two, one))
    vals = four.gather(2, torch.stack((first, second), dim=2).long()).reshape(rows, cols // 2)
    nib = (first | (second << 2)).view(rows, cols // 8, 2)
    return vals.contiguous(), (nib[:, :, 0] | (nib[:, :, 1] << 4)).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    st = {"case": dict(case)}
    m = case["M"]
    if case["op"] == "distill":
        n, k = case["n_vocab"], case["k"]
        z = torch.randn((m, n), generator=g, device="cuda").mul_(2.5)
        t = torch.randn((m, n), generator=g, device="cuda").mul_(0.7).add_(z).topk(k, dim=1)
        st["logits"] = z.to(torch.bfloat16)
        st["teacher"], st["idx"] = t.values.contiguous(), t.indices.to(torch.int32)
        st["dloss"] = torch.full((m,), 1.0 / (m - case["pad"]), device="cuda")
        if case["pad"]:  # padded tokens: no teacher entry, no weight
            st["idx"][m - case["pad"]:] = -1
            st["dloss"][m - case["pad"]:] = 0.0
        if case["pass"] == "backward":  # the forward pass's statistic, kept for the backward pass
            lse = torch.logsumexp(st["logits"].float() / case["tau"], dim=1)
            if case["pad"]:
                lse[m - case["pad"]:] = 0.0
            st["lse"] = lse
        if own and case["pass"] != "forward":
            st["out"] = torch.empty_like(st["logits"])
        return st
    d_out = case["d_out"]
    if case["op"] == "act_grad":
        st["dY"], st["Z"] = normal(m, d_out, std=1e-2), normal(m, d_out, std=1.5)
        return st
    d_in, r = case["d_in"], case["r"]
    st["vals"], st["meta"] = _pack(normal(d_out, d_in, std=0.02))
    st["U"] = normal(d_out, r, std=0.02 / math.sqrt(r)) if r else None
    st["V"] = normal(r, d_in, std=1.0 / math.sqrt(r)) if r else None
    if case["op"] == "dx":
        st["dY"] = normal(m, d_out, std=1e-2)
        if own:
            import sparse_rank_linear_02_b200 as slr
            st["out"] = torch.empty((m, d_in), dtype=torch.bfloat16, device="cuda")
            st["ws"] = torch.empty(max(slr.input_backward_workspace_size(m, d_out, d_in, r), 256), dtype=torch.uint8,
                                   device="cuda")
        return st
    st["X"] = normal(m, d_in)
    st["X"][:, torch.randperm(d_in, generator=g, device="cuda")[: round(0.01 * d_in)]] *= 20  # outlier channels
    st["bias"] = normal(d_out, std=0.1) if case["bias"] else None
    st["residual"] = normal(m, d_out) if case["residual"] else None
    if own:
        import sparse_rank_linear_02_b200 as slr
        st["out"] = torch.empty((m, d_out), dtype=torch.bfloat16, device="cuda")
        st["preact"] = torch.empty_like(st["out"]) if case["preact"] else None
        st["ws"] = torch.empty(max(slr.workspace_size(m, d_out, d_in, r), 256), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- the plain forms and the calls
def _dense(vals, meta):
    """The 2:4 matrix S in fp32 from its packed form."""
    rows, half = vals.shape
    nib = torch.stack((meta & 15, meta >> 4), dim=2).view(rows, half // 2, 1)
    v = vals.float().view(rows, half // 2, 2)
    at = torch.arange(4, device=vals.device, dtype=torch.uint8)
    s = torch.where(at == (nib & 3), v[:, :, :1], 0.0) + torch.where(at == (nib >> 2), v[:, :, 1:], 0.0)
    return s.view(rows, 2 * half)


_C = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":  # 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
        return z / (1.0 + torch.exp(-2.0 * _C * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        s = 1.0 / (1.0 + torch.exp(-2.0 * _C * (z + 0.044715 * z * z * z)))
        return s + z * s * (1.0 - s) * 2.0 * _C * (1.0 + 0.134145 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _teacher(idx, teacher, n, tau):
    """Teacher probabilities over the listed entries (0 where there is none), and their columns."""
    there = (idx >= 0) & (idx < n)
    t = torch.where(there, teacher / tau, -math.inf)
    top = t.max(dim=1, keepdim=True).values
    e = torch.exp(t - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0), torch.where(there, idx, 0).long()


def _distill(st):
    c = st["case"]
    tau = c["tau"]
    z = st["logits"].float() / tau
    p, at = _teacher(st["idx"], st["teacher"], c["n_vocab"], tau)
    some = p.sum(dim=1) > 0
    if c["pass"] == "backward":
        lse = st["lse"]
    else:
        top = z.max(dim=1, keepdim=True).values
        lse = torch.log(torch.exp(z - top).sum(dim=1)) + top[:, 0]
        each = p * (torch.log(torch.where(p > 0, p, 1.0)) - (z.gather(1, at) - lse[:, None]))
        loss = tau * tau * torch.where(p > 0, each, 0.0).sum(dim=1)
        lse = torch.where(some, lse, 0.0)
    if c["pass"] == "forward":
        return [loss, lse]
    w = torch.where(some, tau * st["dloss"], 0.0)[:, None]
    dz = torch.exp(z - lse[:, None]) * w
    dz.scatter_add_(1, at, -p * w)
    dz = torch.where(w != 0, dz, 0.0).to(torch.bfloat16)
    return [dz] if c["pass"] == "backward" else [loss, dz]


def _plain(st):
    c = st["case"]
    if c["op"] == "distill":
        return _distill(st)
    if c["op"] == "act_grad":
        dz = st["dY"].float() * _act_slope(st["Z"].float(), c["act"])
        return [dz.to(torch.bfloat16), dz.sum(dim=0)]
    s = _dense(st["vals"], st["meta"])
    if c["op"] == "dx":
        dy = st["dY"].float()
        dx = dy @ s
        if c["r"]:
            dx += (dy @ st["U"].float()) @ st["V"].float()
        return [dx.to(torch.bfloat16)]
    x = st["X"].float()
    z = x @ s.t()
    if c["r"]:
        z += (x @ st["V"].float().t()) @ st["U"].float().t()
    if c["bias"]:
        z += st["bias"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + st["residual"].float()
    y = y.to(torch.bfloat16)
    return [y, z.to(torch.bfloat16)] if c["preact"] else [y]


def run(st):
    if not own:
        return _plain(st)
    import sparse_rank_linear_02_b200 as slr
    c = st["case"]
    if c["op"] == "forward":
        y = slr.forward_epilogue(st["X"], st["vals"], st["meta"], st["U"], st["V"], bias=st["bias"], act=c["act"],
                                 residual=st["residual"], preact=st["preact"], out=st["out"], workspace=st["ws"])
        return [y, st["preact"]] if c["preact"] else [y]
    if c["op"] == "act_grad":
        return list(slr.epilogue_backward(st["dY"], st["Z"], c["act"]))
    if c["op"] == "dx":
        return [slr.input_backward(st["dY"], st["vals"], st["meta"], st["U"], st["V"], out=st["out"],
                                   workspace=st["ws"])]
    if c["pass"] == "forward":
        return list(slr.distill_forward(st["logits"], st["idx"], st["teacher"], tau=c["tau"]))
    if c["pass"] == "backward":
        return [slr.distill_backward(st["logits"], st["idx"], st["teacher"], st["lse"], st["dloss"], tau=c["tau"],
                                     out=st["out"])]
    return list(slr.distill_loss_grad(st["logits"], st["idx"], st["teacher"], st["dloss"], tau=c["tau"],
                                      out=st["out"]))


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_sparse(st):
    rows, half = st["vals"].shape
    meta = st["meta"].long()
    nib = torch.stack([meta % 16, meta // 16], dim=-1).reshape(rows, half // 2)
    cols = torch.stack([nib % 4, nib // 4], dim=-1) + 4 * torch.arange(half // 2, device=meta.device)[None, :, None]
    s = torch.zeros((rows, 2 * half), dtype=torch.float64, device=meta.device)
    return s.scatter_(1, cols.reshape(rows, half), st["vals"].double())


def _exact_act(z, act, slope):
    if act == "none":
        return torch.ones_like(z) if slope else z
    if act == "relu":
        return torch.heaviside(z, torch.zeros_like(z)) if slope else z.clamp_min(0)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi) if slope else z * cdf
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        if not slope:
            return z * torch.sigmoid(2 * u)
        du = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
        return torch.sigmoid(2 * u) + 2 * z * torch.sigmoid(2 * u) * torch.sigmoid(-2 * u) * du
    s = torch.sigmoid(z)
    return s + z * s * torch.sigmoid(-z) if slope else z * s


def _exact_distill(st):
    c = st["case"]
    m, n, tau = c["M"], c["n_vocab"], c["tau"]
    dev = st["logits"].device
    loss = torch.zeros(m, dtype=torch.float64, device=dev)
    lse = torch.zeros(m, dtype=torch.float64, device=dev)
    dz = torch.zeros((m, n), dtype=torch.float64, device=dev) if c["pass"] != "forward" else None
    for lo in range(0, m, 512):  # tokens are independent: blocks bound the memory
        rows = [i for i in range(lo, min(lo + 512, m)) if i < m - c["pad"]]
        if not rows:
            continue
        sl = slice(rows[0], rows[-1] + 1)
        logq = torch.log_softmax(st["logits"][sl].double() / tau, dim=1)
        logp = torch.log_softmax(st["teacher"][sl].double() / tau, dim=1)
        at = st["idx"][sl].long()
        loss[sl] = tau ** 2 * (logp.exp() * (logp - logq.gather(1, at))).sum(dim=1)
        lse[sl] = torch.logsumexp(st["logits"][sl].double() / tau, dim=1)
        if dz is not None:
            w = tau * st["dloss"][sl].double()[:, None]
            if c["pass"] == "backward":  # q from the statistic that the call is given
                logq = st["logits"][sl].double() / tau - st["lse"][sl].double()[:, None]
            dz[sl] = logq.exp().scatter_add(1, at, -logp.exp()) * w
    if c["pass"] == "forward":
        return [loss, lse]
    return [dz] if c["pass"] == "backward" else [loss, dz]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "distill":
        return _exact_distill(st)
    if case["op"] == "act_grad":
        dz = st["dY"].double() * _exact_act(st["Z"].double(), case["act"], True)
        return [dz, dz.sum(dim=0)]
    w = _exact_sparse(st)
    if case["r"]:
        w += st["U"].double() @ st["V"].double()
    if case["op"] == "dx":
        return [st["dY"].double() @ w]
    z = st["X"].double() @ w.t()
    if case["bias"]:
        z = z + st["bias"].double()
    y = _exact_act(z, case["act"], False)
    if case["residual"]:
        y = y + st["residual"].double()
    return [y, z] if case["preact"] else [y]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    m = case["M"]
    if case["op"] == "distill":
        n, k = case["n_vocab"], case["k"]
        live = m - case["pad"]
        read = 2 * live * n + 8 * m * k
        wrote = 4 * m if case["pass"] != "backward" else 0
        wrote += 4 * m if case["pass"] == "forward" else 2 * m * n
        read += {"forward": 0, "backward": 8 * m, "step": 4 * m}[case["pass"]]
        return {"bytes": read + wrote, "flops": (4 if case["pass"] == "forward" else 6) * live * n}
    d_out = case["d_out"]
    if case["op"] == "act_grad":
        return {"bytes": 6 * m * d_out + 4 * d_out, "flops": 12 * m * d_out}
    d_in, r = case["d_in"], case["r"]
    layer = d_out * d_in + d_out * d_in // 8 + 2 * r * (d_out + d_in)  # kept values, metadata, factors
    flops = m * d_out * d_in + 2 * m * r * (d_out + d_in)              # two kept weights of four
    ends = 2 * m * (d_in + d_out)
    if case["op"] == "forward":
        ends += 2 * d_out * case["bias"] + 2 * m * d_out * (case["residual"] + case["preact"])
    return {"bytes": layer + ends, "flops": flops}
