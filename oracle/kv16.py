"""The 16-bit K/V cache operators in numpy, from their definitions (include/llm_ops.h), in 64 bits.

Pools are float arrays [pages][Hkv][16][d] that hold the 16-bit numbers' values; what an operator copies is copied.
"""
import numpy as np

from .kv8 import PAGE, sequences


def slots(pages, n):
    """(page, place in it) of the first n slots of these pages."""
    t = np.arange(n)
    return np.asarray(pages, np.int64)[t // PAGE], t % PAGE


def rotate(x, gain, eps, base, axis, pos):
    """RMS norm (gain None: none) and rotation: x [rows][heads][d], axis [d/2], pos [axes][rows] -> float64."""
    x = x.astype(np.float64)
    d = x.shape[-1]
    if gain is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * gain.astype(np.float64)
    ang = np.asarray(pos, np.float64)[np.asarray(axis)].T * base ** (-2.0 * np.arange(d // 2) / d)
    co, si = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([a * co - b * si, b * co + a * si], -1)


def _values(pool, pages, n, g):
    page, at = slots(pages, n)
    return pool[page, g, at].astype(np.float64)


def attention(k_pool, v_pool, table, row_start, kv_len, q, prefix=None):
    """q [rows][Hq][d]; prefix: (table, len, seq_start) -> out, lse, and per (row, head) what bounds on the error are made of:
    the weighted sum of |V| (as out) and the largest sum of |q_i k_i| / sqrt(d) over the keys."""
    rows, Hq, d = q.shape
    Hkv = k_pool.shape[1]
    out, absv = np.zeros((rows, Hq, d)), np.zeros((rows, Hq, d))
    lse, absqk = np.full((rows, Hq), -np.inf), np.zeros((rows, Hq))
    for b, row0, n, kv in sequences(row_start, kv_len):
        front, p = None, 0
        if prefix is not None:
            for g in range(len(prefix[1])):
                if prefix[2][g] <= b < prefix[2][g + 1]:
                    front, p = prefix[0][g], int(prefix[1][g])
        if n == 0:
            continue
        own = np.arange(p + kv)[None, :] - p
        hidden = (own >= 0) & (own > np.arange(kv - n, kv)[:, None])
        for g in range(Hkv):
            K, V = (_values(pool, table[b], kv, g) for pool in (k_pool, v_pool))
            if p:
                K, V = np.concatenate([_values(k_pool, front, p, g), K]), np.concatenate([_values(v_pool, front, p, g), V])
            for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                x = q[row0:row0 + n, h].astype(np.float64)
                with np.errstate(all="ignore"):
                    s = np.where(hidden, -np.inf, x @ K.T / np.sqrt(d))
                    size = np.where(hidden, 0, np.abs(x) @ np.abs(K).T / np.sqrt(d))
                    top = s.max(-1, initial=-np.inf)
                    w = np.exp(s - np.where(np.isneginf(top), 0, top)[:, None])
                    total = w.sum(-1)
                    lse[row0:row0 + n, h] = top + np.log(total)
                    w = w / np.where(total == 0, 1, total)[:, None]
                    live = ~hidden.all(0)
                    out[row0:row0 + n, h] = w[:, live] @ V[live]
                    absv[row0:row0 + n, h] = w[:, live] @ np.abs(V[live])
                absqk[row0:row0 + n, h] = size.max(-1, initial=0)
    return out, lse, absv, absqk


def weigh(k_pool, table, row_start, kv_len, q, lse, keep, scores):
    """-> the new scores in float64, and the sum over a token's terms of term * (sum of |q_i k_i| / sqrt(d) + |lse| + 1)."""
    Hq, d = q.shape[1:]
    Hkv = k_pool.shape[1]
    new, size = scores.astype(np.float64), np.zeros(scores.shape)
    for b, row0, n, kv in sequences(row_start, kv_len):
        if n == 0:
            continue
        hidden = np.arange(kv)[None, :] > np.arange(kv - n, kv)[:, None]
        first = max(0, kv - n)
        new[b, :, first:kv] = 0
        new[b, :, :first] = keep * new[b, :, :first] if keep else 0
        for g in range(Hkv):
            K = _values(k_pool, table[b], kv, g)
            for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                x, y = q[row0:row0 + n, h].astype(np.float64), lse[row0:row0 + n, h].astype(np.float64)[:, None]
                with np.errstate(all="ignore"):
                    w = np.where(hidden | np.isneginf(y), 0, np.exp(x @ K.T / np.sqrt(d) - y))
                    new[b, g, :kv] += w.sum(0)
                    size[b, g, :kv] += np.where(w > 0, w * (np.abs(x) @ np.abs(K).T / np.sqrt(d) + np.abs(y) + 1), 0).sum(0)
    return new, size


def choose(scores, n, budget, n_first, n_last):
    """The slots that stay of a sequence and head, ascending."""
    if n <= budget:
        return np.arange(n)
    s = np.where(np.isnan(scores[:n]), -np.inf, scores[:n].astype(np.float64))
    nan = np.isnan(scores[:n])
    middle = np.arange(n_first, n - n_last)
    order = sorted(middle, key=lambda i: (nan[i], -s[i], i))[:budget - n_first - n_last]
    return np.concatenate([np.arange(n_first), np.sort(np.asarray(order, np.int64)), np.arange(n - n_last, n)]).astype(np.int64)


def evict(pools, table, kv_len, budget, n_first, n_last, scores, scores_out, kept):
    """Changes pools (a list of arrays), scores_out and kept; -> new_len."""
    for b, n in enumerate(int(x) for x in kv_len):
        for g in range(scores.shape[1]):
            stay = choose(scores[b, g], n, budget, n_first, n_last)
            kept[b, g, :len(stay)] = stay
            scores_out[b, g, :len(stay)] = scores[b, g][stay]
            page, at = slots(table[b], n)
            for pool in pools:
                pool[page[:len(stay)], g, at[:len(stay)]] = pool[page[stay], g, at[stay]]
    return np.minimum(kv_len, budget)
