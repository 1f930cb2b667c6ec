"""Plain 64-bit forms of the expert operators on numpy arrays, for the tests:
one expert, or one assignment, at a time."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24   # unit roundoff of fp32


def order_ref(ids, E):
    """(offsets, source, slot) by counting, in Python integers."""
    T, k = ids.shape
    offsets, source = [0], []
    slot = np.full((T, k), -1, np.int64)
    for e in range(E):
        for t, j in np.argwhere(ids == e):
            slot[t, j] = len(source)
            source.append(t * k + j)
        offsets.append(len(source))
    source += [-1] * (T * k - len(source))
    return np.array(offsets), np.array(source, dtype=np.int64).reshape(-1), slot


def gather_ref(x, source, k):
    out = np.zeros((len(source), x.shape[1]))
    kept = source >= 0
    out[kept] = x[source[kept] // k]
    return out


def combine_ref(ys, slot, w):
    """(y, sum of |terms|)."""
    T, k = slot.shape
    y = np.zeros((T, ys.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            if slot[t, j] >= 0:
                term = (1.0 if w is None else float(w[t, j])) * ys[slot[t, j]]
                y[t] += term
                mag[t] += np.abs(term)
    return y, mag


def combine_grad_ref(dy, ys, slot, w):
    """(dys, dw, sum of |terms| of dw)."""
    T, k = slot.shape
    dys = np.zeros((T * k, dy.shape[1]))
    dw = np.zeros((T, k))
    mag = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            s = slot[t, j]
            if s >= 0:
                dys[s] = (1.0 if w is None else float(w[t, j])) * dy[t]
                dw[t, j] = np.dot(dy[t], ys[s])
                mag[t, j] = np.dot(np.abs(dy[t]), np.abs(ys[s]))
    return dys, dw, mag


def _round(a, dtype):
    return torch.from_numpy(np.asarray(a, dtype=np.float64)).to(dtype).double().numpy()


def within(got, want, bound, dtype) -> bool:
    """Whether every element of got, of type dtype, can come from a value
    within `bound` of want by one rounding: rounding is monotonic, so got
    lies between the rounded ends of that interval."""
    got = got.detach().cpu().double().numpy()
    return bool(np.all((got >= _round(want - bound, dtype)) & (got <= _round(want + bound, dtype))))
