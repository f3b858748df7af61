"""The layer's epilogue (bias, activation, residual), its gradient and the
gradient of the layer's input, in fp64.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py): used by the tests and the
smoke check, never by the product path.

    Z = X W'^T + b,  W' = S + U V          Y = act(Z) + R
    dZ = dY act'(Z)      db_j = sum_m dZ_mj      dX = dZ W'

The activations are written from their definitions: relu, z Phi(z), its tanh
form and z sigma(z).  Each function also returns the sums of magnitudes from
which the tests derive their tolerances.
"""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erfc

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def act(z: np.ndarray, kind: str) -> np.ndarray:
    if kind == "none":
        return z
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "gelu":
        return 0.5 * z * erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * _sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if kind == "silu":
        return z * _sigmoid(z)
    raise ValueError(kind)


def act_slope(z: np.ndarray, kind: str) -> np.ndarray:
    if kind == "none":
        return np.ones_like(z)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        u = c * (z + 0.044715 * z ** 3)
        return _sigmoid(u) + z * _sigmoid(u) * _sigmoid(-u) * c * (1.0 + 3 * 0.044715 * z ** 2)
    if kind == "silu":
        return _sigmoid(z) + z * _sigmoid(z) * _sigmoid(-z)
    raise ValueError(kind)


def dense(vals: np.ndarray, meta: np.ndarray) -> np.ndarray:
    """S [d_out, d_in] in fp64 from bf16 bit patterns and index nibbles."""
    rows, half = vals.shape
    v = (np.ascontiguousarray(vals, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    nib = np.stack([meta & 15, meta >> 4], axis=-1).reshape(rows, -1)[:, : half // 2].astype(np.int64)
    s = np.zeros((rows, half // 2, 4))
    r, g = np.indices(nib.shape)
    s[r, g, nib & 3] = v[:, 0::2]
    s[r, g, nib >> 2] = v[:, 1::2]
    return s.reshape(rows, 2 * half)


def forward(X, S, U, V, bias, kind, R):
    """(Y, Z, |X| |S|^T + |T| |U|^T + |b|, |T| |U|^T) in fp64, T = X V^T; U, V, bias and R may be None."""
    Z, B = X @ S.T, np.abs(X) @ np.abs(S).T
    BT = np.zeros_like(Z)
    if U is not None:
        Z = Z + (X @ V.T) @ U.T
        BT = (np.abs(X) @ np.abs(V).T) @ np.abs(U).T
        B = B + BT
    if bias is not None:
        Z, B = Z + bias, B + np.abs(bias)
    Y = act(Z, kind)
    return (Y if R is None else Y + R), Z, B, BT


def input_backward(dY, S, U, V):
    """(dX, its bound |dY| |S| + |dY| |U| |V|, the second term alone) in fp64."""
    dX, B = dY @ S, np.abs(dY) @ np.abs(S)
    BT = np.zeros_like(dX)
    if U is not None:
        dX = dX + (dY @ U) @ V
        BT = (np.abs(dY) @ np.abs(U)) @ np.abs(V)
        B = B + BT
    return dX, B, BT
