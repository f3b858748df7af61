"""Distillation of a student's logits from a teacher's top logits, in fp64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py): used by the tests and the
smoke check, never by the product path.

Per token: p the softmax over the teacher's listed logits t / tau (an entry
whose column is outside the vocabulary or whose logit is -inf is not there), q
the softmax of the student's z / tau,

    loss = tau^2 KL(p || q)        dloss/dz_v = tau (q_v - sum of p_j listed at v)

written row by row from that definition.  A token without entries has loss 0,
lse 0 and a zero gradient.
"""
from __future__ import annotations

import numpy as np


def distill(z: np.ndarray, idx: np.ndarray, t: np.ndarray, tau: float):
    """(loss [M], lse [M], dz [M, n], |log p - log q| weighted by p [M]) in fp64."""
    M, n = z.shape
    loss, lse, dz, spread = np.zeros(M), np.zeros(M), np.zeros((M, n)), np.zeros(M)
    for m in range(M):
        at = [(int(i), float(x) / tau) for i, x in zip(idx[m], t[m]) if 0 <= i < n and x != -np.inf]
        if not at:
            continue
        cols, x = np.array([i for i, _ in at]), np.array([x for _, x in at])
        logp = x - (x.max() + np.log(np.exp(x - x.max()).sum()))
        p = np.exp(logp)
        y = z[m] / tau
        logs = np.log(np.exp(y - y.max()).sum())
        lse[m] = y.max() + logs
        logq = (y - y.max()) - logs   # not y - lse: next to the type's lowest values lse has no digits left for logs
        term = np.where(p > 0, p * (logp - logq[cols]), 0.0)
        loss[m] = tau ** 2 * term.sum()
        spread[m] = np.abs(term).sum()
        g = np.exp(logq)
        for i, pj in zip(cols, p):
            g[i] -= pj
        dz[m] = tau * g
    return loss, lse, dz, spread
