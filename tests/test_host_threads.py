"""Calls from several host threads at once.  On the CPU: whatever a function of the
library keeps between calls is atomic, behind a lock or set up once (read from the
sources, since a race shows by chance alone).  On the GPU: the operators' first calls
and later ones, made from four threads on streams of their own."""
import glob
import os
import re
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_rank_linear_02_b200", "csrc")
KEPT = re.compile(r"^ +static (?!constexpr\b|const\b|inline\b|std::mutex\b|std::once_flag\b|std::atomic\b)\w", re.M)


def functions():
    """(file, text) of every top-level function or class of the host and device sources."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            for block in re.split(r"^}", f.read(), flags=re.M):
                yield os.path.basename(path), block


def test_what_is_kept_between_calls_is_safe():
    kept = [(f, b) for f, b in functions() if KEPT.search(b)]
    assert kept   # the device check, the plans
    for file, block in kept:
        assert re.search(r"std::lock_guard|std::call_once", block), f"{file}:{block[-400:]}"


CHILD = """
import threading, torch
import sparse_rank_linear_02_b200 as slr

def layer(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    W, U, V, X, dY = n(1032, 512), n(1032, 64), n(64, 512), n(300, 512), n(300, 1032)
    idx = torch.randint(0, 1032, (300, 8), generator=g, device="cuda", dtype=torch.int32)
    t, w = torch.randn((300, 8), generator=g, device="cuda"), torch.rand(300, generator=g, device="cuda")
    return W, U, V, X, dY, idx, t, w

def step(W, U, V, X, dY, idx, t, w):
    vals, meta = slr.pack_2to4(W)
    Z = torch.empty_like(dY)
    Y = slr.forward_epilogue(X, vals, meta, U, V, act="gelu", residual=dY, preact=Z)
    dZ, db = slr.epilogue_backward(dY, Z, "gelu")
    return [Y, Z, dZ, db, slr.input_backward(dZ, vals, meta, U, V), *slr.lora_backward(X, dZ, U, V),
            *slr.distill_loss_grad(Y, idx, t, w)]

ops, got, errors = [layer(s) for s in range(4)], [None] * 4, []
torch.cuda.synchronize()
start = threading.Barrier(4)

def work(i):
    try:
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()) as s:
            start.wait()
            got[i] = [step(*ops[i]) for _ in range(8)]
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
slr.check_kernel_error()
for i in range(4):
    want = step(*ops[i])
    assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want)), i
print("threads ok")
"""


@pytest.mark.gpu
def test_first_and_later_calls_from_four_threads():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
