"""The serving step in numpy float64: the new rows and queries, and the attention
over a sequence's rows, straight from the formulas in include/leyline_step.h.
Shares no code with the library."""

from __future__ import annotations

import numpy as np


def angles(positions, rot: int, base: float) -> np.ndarray:
    """[tokens][rot / 2] float64 angles."""
    j = np.arange(rot // 2, dtype=np.float64)
    return np.asarray(positions, np.float64)[:, None] * np.power(base, -2.0 * j / rot)[None]


def rotate(x: np.ndarray, ang: np.ndarray, pairing: int) -> np.ndarray:
    """x [tokens][heads][rot] turned by each token's angles (pairing 0: pairs
    (2j, 2j + 1); 1: pairs (j, j + rot / 2))."""
    z = np.exp(1j * ang)[:, None]
    h = x.shape[-1] // 2
    if pairing == 0:
        y = (x[..., 0::2] + 1j * x[..., 1::2]) * z
        out = np.empty_like(x)
        out[..., 0::2], out[..., 1::2] = y.real, y.imag
        return out
    y = (x[..., :h] + 1j * x[..., h:]) * z
    return np.concatenate([y.real, y.imag], -1)


def norm(x: np.ndarray, w, eps: float) -> np.ndarray:
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w


def heads(x, w, eps, ang, pairing, rot=None):
    """(result, size) of normed and rotated heads [tokens][heads][dim]; size bounds
    the magnitudes that entered each value's rotation."""
    y = norm(x, w, eps)
    rot = y.shape[-1] if rot is None else rot
    z = y.copy()
    z[..., :rot] = rotate(y[..., :rot], ang, pairing)
    size = np.abs(y)
    h = rot // 2
    if pairing == 0:
        s = size[..., 0:rot:2] + size[..., 1:rot:2]
        size[..., 0:rot:2], size[..., 1:rot:2] = s, s
    else:
        s = size[..., :h] + size[..., h:rot]
        size[..., :h], size[..., h:rot] = s, s
    return z, size


def attend(q, k, v, first: int, scale: float, causal: bool = True, window: int = 0):
    """One head of one sequence: q [n][dk], k [rows][dk], v [rows][dv]; query i is
    row first + i.  Returns (out, lse, weight, slack): weight is sum p |v|, slack
    bounds scale * sum |q| |k| over the rows seen."""
    n, rows = q.shape[0], k.shape[0]
    out = np.zeros((n, v.shape[1]))
    weight = np.zeros_like(out)
    lse = np.full(n, -np.inf)
    slack = np.zeros(n)
    for i in range(n):
        hi = first + i + 1 if causal else rows
        lo = max(0, hi - window) if window else 0
        if hi <= lo:
            continue
        s = scale * (k[lo:hi] @ q[i])
        m = s.max()
        p = np.exp(s - m)
        total = p.sum()
        out[i] = (p @ v[lo:hi]) / total
        weight[i] = (p @ np.abs(v[lo:hi])) / total
        lse[i] = m + np.log(total)
        slack[i] = abs(scale) * (np.abs(k[lo:hi]) @ np.abs(q[i])).max()
    return out, lse, weight, slack
