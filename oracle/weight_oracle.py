"""Eviction by attention weight and the trainer's attention in numpy float64,
straight from the formulas in include/leyline_weight.h and include/leyline_train.h.
Shares no code with the library."""

from __future__ import annotations

import numpy as np


def capped(x: np.ndarray, cap: float) -> np.ndarray:
    return cap * np.tanh(x / cap) if cap else x


def scores(q, k, scale: float, cap: float = 0.0):
    """(scores [n][rows], slack): slack bounds |scale| * sum |q| |k| of each."""
    return capped(scale * (q @ k.T), cap), abs(scale) * (np.abs(q) @ np.abs(k).T)


def step_seen(n: int, rows: int, first: int, causal: bool = True, window: int = 0) -> np.ndarray:
    """[n][rows]: query i is row first + i."""
    own, j = first + np.arange(n)[:, None], np.arange(rows)[None]
    seen = j <= own if causal else np.ones((n, rows), bool)
    return seen & (j > own - window) if window else seen


def death_seen(death: np.ndarray) -> np.ndarray:
    """[T][T]: query q sees key k iff k <= q < death[k]."""
    t = np.arange(len(death))
    return (t[None] <= t[:, None]) & (t[:, None] < np.asarray(death, np.int64)[None])


def softmax(x, seen):
    """(weights, lse) of the seen scores of each row; none seen: zeros and -inf."""
    x = np.where(seen, x, -np.inf)
    m = x.max(-1, keepdims=True, initial=-np.inf)
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        p = np.exp(x - m)
        total = p.sum(-1, keepdims=True)
        return p / np.where(total > 0, total, 1.0), (m + np.log(total))[:, 0]


def attend(q, k, v, seen, scale: float, cap: float = 0.0):
    """One head: (out, lse, weight, slack), weight = sum p |v|, slack = the largest
    |scale| sum |q| |k| among a query's seen rows."""
    x, s = scores(q, k, scale, cap)
    p, lse = softmax(x, seen)
    return p @ v, lse, p @ np.abs(v), np.where(seen, s, 0.0).max(-1, initial=0.0)


def weigh(q, k, lse, seen, scale: float, cap: float = 0.0):
    """One head's part of the weights [rows], its tolerance's parts: sum p * slack and
    sum p * (1 + |score| + |lse|)."""
    x, s = scores(q, k, scale, cap)
    live = seen & (lse != -np.inf)[:, None]
    ls = np.where(np.isfinite(lse), lse, 0.0)[:, None]
    p = np.where(live, np.exp(np.where(live, x - ls, 0.0)), 0.0)
    return p.sum(0), (p * s).sum(0), (p * (1 + np.abs(x) + np.abs(ls))).sum(0)


def keep_heaviest(weights, budget: int, sinks: int, recent: int) -> np.ndarray:
    """Keep bytes of one sequence's rows (weights: float32 [rows])."""
    n = len(weights)
    keep = np.zeros(n, np.uint8)
    keep[:min(sinks, n)] = 1
    keep[max(0, n - recent):] = 1
    rest = [i for i in range(n) if not keep[i]]
    w = np.asarray(weights, np.float64)
    rest.sort(key=lambda i: (not np.isnan(w[i]), 0.0 if np.isnan(w[i]) else -w[i], i))
    keep[rest[:max(0, min(budget, n) - int(keep.sum()))]] = 1
    return keep


def gradients(q, k, v, dout, seen, scale: float, cap: float = 0.0):
    """One head's (dq, dk, dv) in the order of the formulas."""
    raw = scale * (q @ k.T)
    p, _ = softmax(capped(raw, cap), seen)
    dp = dout @ v.T
    delta = (dout * (p @ v)).sum(-1, keepdims=True)
    ds = p * (dp - delta) * scale
    if cap:
        ds = ds * (1 - np.tanh(raw / cap) ** 2)
    return ds @ k, ds.T @ q, p.T @ dout
