"""Plain float64 CPU oracle of the paged key/value cache and of the attention that reads it
(test infrastructure, like the rest of this package).

Cache: [pages, kv heads, page size, head dim] for keys and the same for values. Slot =
page * page size + offset. An 8-bit cache holds e4m3 codes c that stand for c * scale[kv head].

Attention of one sequence: n query tokens, the last n of its kv cached tokens. For query head h
(kv head h // group) over the visible tokens j:
    z_j = scale q.k_j  (softcap tanh(z_j / softcap) when softcap > 0)
    lse = log sum exp z_j,  out = sum exp(z_j - lse) v_j;  nothing visible: out = 0, lse = -inf.
"""
from __future__ import annotations

import numpy as np


def visible_tree(n: int, kv: int, mask_words) -> np.ndarray:
    """[n, kv] booleans: all of the first kv - n tokens, and token kv - n + b where bit b of the
    row's word is set; mask_words None: a chain."""
    see = np.zeros((n, max(kv, 0)), bool)
    ctx = kv - n
    for i in range(n):
        see[i, :max(ctx, 0)] = True
        for b in range(n):
            j = ctx + b
            if j < 0:
                continue
            see[i, j] = b <= i if mask_words is None else bool((int(mask_words[i]) >> b) & 1)
    return see


def visible_prefill(n: int, kv: int, prefix: int) -> np.ndarray:
    """[n, kv] booleans: token j for row i when j <= kv - n + i or j < prefix."""
    j = np.arange(max(kv, 0))[None, :]
    i = np.arange(n)[:, None]
    return (j <= kv - n + i) | (j < prefix)


def visible_window(n: int, kv: int, window: int, sinks: int) -> np.ndarray:
    """[n, kv] booleans: token j for row i, at position p = kv - n + i, when j <= p and (p - j < window or j < sinks)."""
    j = np.arange(max(kv, 0))[None, :]
    p = kv - n + np.arange(n)[:, None]
    return (j <= p) & ((p - j < window) | (j < sinks))


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, see: np.ndarray, scale: float, softcap: float = 0.0):
    """One sequence: q [n, Hq, D], k and v [kv, Hkv, D], see [n, kv] -> out [n, Hq, D], lse [n, Hq],
    and for error bounds the weighted mean of |v| [n, Hq, D] and the largest sum |q_d k_d| * scale [n, Hq]."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    group = Hq // Hkv
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, dot = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    some = see.any(axis=1)
    if not some.any():
        return out, lse, mag, dot
    for h in range(Hq):
        kh, vh = np.asarray(k[:, h // group], np.float64), np.asarray(v[:, h // group], np.float64)
        qh = np.asarray(q[:, h], np.float64)
        z = scale * (qh @ kh.T)
        if softcap > 0:
            z = softcap * np.tanh(z / softcap)
        z = np.where(see, z, -np.inf)
        m = np.where(some, z.max(axis=1, initial=-np.inf), 0.0)
        p = np.exp(z - m[:, None])
        total = np.where(some, p.sum(axis=1), 1.0)
        w = p / total[:, None]
        out[:, h] = w @ vh
        mag[:, h] = w @ np.abs(vh)
        lse[:, h] = np.where(some, m + np.log(total), -np.inf)
        dot[:, h] = np.where(see, scale * (np.abs(qh) @ np.abs(kh).T), 0.0).max(axis=1)
    return out, lse, mag, dot


def usage(q: np.ndarray, k: np.ndarray, see: np.ndarray, lse: np.ndarray, scale: float, softcap: float = 0.0):
    """One sequence: q [n, Hq, D], k [kv, Hkv, D], see [n, kv], lse [n, Hq] -> [Hkv, kv] sums over the tokens and the heads
    of a kv head of exp(z - lse), and for error bounds the same sums with every weight times the row's largest
    sum |q_d k_d| * scale."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    group = Hq // Hkv
    out, spread = np.zeros((Hkv, see.shape[1])), np.zeros((Hkv, see.shape[1]))
    if n == 0 or see.shape[1] == 0:
        return out, spread
    for h in range(Hq):
        kh, qh = np.asarray(k[:, h // group], np.float64), np.asarray(q[:, h], np.float64)
        z = scale * (qh @ kh.T)
        if softcap > 0:
            z = softcap * np.tanh(z / softcap)
        top = np.where(np.isneginf(lse[:, h]), np.inf, lse[:, h]).astype(np.float64)
        p = np.where(see, np.exp(z - top[:, None]), 0.0)
        dot = np.where(see, scale * (np.abs(qh) @ np.abs(kh).T), 0.0).max(axis=1)
        out[h // group] += p.sum(axis=0)
        spread[h // group] += (p * dot[:, None]).sum(axis=0)
    return out, spread


def kept_tokens(usage_row: np.ndarray, n: int, budget: int, sinks: int, recent: int) -> np.ndarray:
    """The places, ascending, of the `budget` of n tokens that stay: the first `sinks`, the last `recent`, and of the rest
    those of largest usage, equal ones by place; NaN below everything."""
    middle = list(range(sinks, n - recent))
    value = [(-np.inf, 0) if np.isnan(usage_row[j]) else (usage_row[j], 1) for j in middle]
    best = sorted(range(len(middle)), key=lambda i: (-value[i][0], -value[i][1], middle[i]))
    chosen = [middle[i] for i in best[:budget - sinks - recent]]
    return np.array(sorted(list(range(sinks)) + chosen + list(range(n - recent, n))), np.int32)
