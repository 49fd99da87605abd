"""CPU oracle for the scores of given tokens with their alternatives, their
gradient, and the slots that a cache keeps.

TEST INFRASTRUCTURE ONLY, like qrita_oracle: nothing on the product path
imports it, and it shares no code with the CUDA library.

Plain fp64 definitions, one row at a time (include/qrita.h states the contract):

* ``scores_row``: log-probabilities, rank, entropy and top alternatives;
* ``scores_grad_row``: the gradient of their weighted sum;
* ``cache_weights``: attention weights of queries on the slots of a cache;
* ``kept_order``: the order in which a cache keeps its slots.

Pins: tests/test_oracle_scores.py.
"""

from __future__ import annotations

import numpy as np


def _log_softmax(x, kept, inv_t):
    """(log p over all ids, -inf off the kept set; whether the row is NaN)."""
    logs = np.full(x.shape[0], -np.inf)
    xs = x[kept]
    if xs.size == 0 or np.isneginf(xs).all():
        return logs, False
    if np.isnan(xs).any() or np.isposinf(xs).any():
        return logs, True
    y = (xs - xs.max()) * inv_t
    logs[kept] = y - np.log(np.exp(y).sum())
    logs[kept & np.isneginf(x)] = -np.inf
    return logs, False


def _entropy(logs):
    with np.errstate(invalid="ignore"):
        p = np.exp(logs)
        return float(-np.where(p > 0, p * logs, 0.0).sum())


def scores_row(x, mask, tokens, inv_t=1.0, top=0):
    """(logp [M], rank of the first token, entropy, top ids, top logp)."""
    x = np.asarray(x, np.float64)
    V = x.shape[0]
    kept = np.ones(V, bool) if mask is None else np.asarray(mask) != 0
    logs, nan = _log_softmax(x, kept, inv_t)
    inside = [0 <= t < V for t in tokens]
    if nan:
        return (np.array([np.nan if i else 0.0 for i in inside]), -1, np.nan, np.full(top, -1), np.full(top, np.nan))
    logp = np.array([logs[t] if i else 0.0 for t, i in zip(tokens, inside)])
    # kept ids with p > 0 in the stable descending order (a logit of -inf has p = 0)
    live = np.flatnonzero(kept & (x > -np.inf))
    ids = live[np.argsort(-x[live], kind="stable")]
    rank = -1
    if len(tokens) and inside[0] and logs[tokens[0]] > -np.inf:
        rank = int(np.flatnonzero(ids == tokens[0])[0])
    first = ids[:top].tolist()
    pad = top - len(first)
    return (logp, rank, _entropy(logs), np.array(first + [-1] * pad),
            np.array([logs[i] for i in first] + [-np.inf] * pad))


def scores_grad_row(x, mask, ids, g, h=0.0, inv_t=1.0):
    """Gradient of sum_i g_i log p(ids_i) + h H with respect to x; also the sum of
    the magnitudes of its terms."""
    x = np.asarray(x, np.float64)
    V = x.shape[0]
    kept = np.ones(V, bool) if mask is None else np.asarray(mask) != 0
    logs, nan = _log_softmax(x, kept, inv_t)
    out, size = np.zeros(V), np.zeros(V)
    some = any(v != 0 for t, v in zip(ids, g) if 0 <= t < V) or h != 0
    if not some:
        return out, size
    if nan:
        out[kept] = np.nan
        return out, size
    p = np.exp(logs)
    for t, v in zip(ids, g):
        if 0 <= t < V and logs[t] > -np.inf:
            out[t] += v
            size[t] += abs(v)
    out, size = out - out.sum() * p, size + size.sum() * p
    if h != 0:
        H = _entropy(logs)
        inner = np.where(p > 0, np.where(p > 0, logs, 0.0) + H, 0.0)
        out -= h * p * inner
        size += abs(h) * p * (np.abs(np.where(p > 0, logs, 0.0)) + H)
    return out * inv_t, size * inv_t


def cache_weights(q, k, positions, length, seen, scale):
    """sum over queries of softmax over visible slots: q [T, G, D], k [S, D] of one
    kv head, positions [S]. Returns [length]."""
    T, G, _ = q.shape
    total = np.zeros(length)
    for t in range(T):
        see = np.asarray(positions[:length]) <= seen - T + t
        if not see.any():
            continue
        for g in range(G):
            s = (k[:length].astype(np.float64) @ q[t, g].astype(np.float64)) * scale
            s = s[see]
            if np.isnan(s).any() or np.isposinf(s).any():
                total[see] = np.nan
                continue
            if np.isneginf(s).all():
                continue
            e = np.exp(s - s.max())
            total[see] += e / e.sum()
    return total


def kept_order(weights, positions, length, seen, sink, recent):
    """The slots [0, length) in the order in which they are kept: protected ones
    (positions below sink, or among the last `recent` seen) first, then by weight
    (larger first, NaN last), equal ones by slot."""
    def key(i):
        p = positions[i]
        guarded = p < sink or p >= seen - recent
        w = float(weights[i])
        return (not guarded, np.isnan(w), 0.0 if np.isnan(w) else -w, i)

    return sorted(range(length), key=key)
