"""Plain 64-bit forms of the projections on numpy arrays, one group at a time,
and the error that fp32 arithmetic may leave, for the tests."""
from __future__ import annotations

import numpy as np

from expert_ref import U32

C = np.sqrt(2 / np.pi)


def act(name, g):
    with np.errstate(all="ignore"):
        if name == "silu":
            return g / (1 + np.exp(-g))
        if name == "gelu_tanh":
            return 0.5 * g * (1 + np.tanh(C * (g + 0.044715 * g ** 3)))
    return np.maximum(g, 0) if name == "relu" else g


def slope(name, g):
    if name == "silu":
        s = 1 / (1 + np.exp(-g))
        return s * (1 + g * (1 - s))
    if name == "gelu_tanh":
        t = np.tanh(C * (g + 0.044715 * g ** 3))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * C * (1 + 3 * 0.044715 * g * g)
    return (g > 0).astype(float) if name == "relu" else np.ones_like(g)


def act_error(g):
    """Of act in fp32: exp and tanh are a few units off (at most 4 units of
    values below 2), and at most 12 roundings of values below 1 + |g| follow."""
    return 16 * U32 * (1 + np.abs(g))


def slope_error(g):
    """Of the slope in fp32: 1 - s and 1 - t^2 are off by some units of 1 (8),
    times g (and 0.134 g^3 for gelu); the rest as act_error."""
    return act_error(g) + 16 * U32 * np.abs(g) * (1 + 0.15 * g * g)


def products(X, W, sizes, lead=0):
    """X's rows times their group's matrix; rows of no group zero."""
    out = np.zeros((X.shape[0], W.shape[2]))
    at = lead
    for g, n in enumerate(sizes):
        out[at:at + n] = X[at:at + n] @ W[g]
        at += n
    return out


def in_group(S, sizes, lead=0):
    rows = np.zeros(S, bool)
    rows[lead:lead + sum(sizes)] = True
    return rows


def adapted(X, W, A, B, sizes, scales=None, lead=0):
    """(Y, U)."""
    U = products(X, A.transpose(0, 2, 1), sizes, lead)
    if scales is not None:
        U[lead:lead + sum(sizes)] *= np.repeat(scales, sizes)[:, None]
    return X @ W + products(U, B, sizes, lead), U
