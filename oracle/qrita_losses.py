"""CPU oracle for the losses over rows of logits and their gradients.

TEST INFRASTRUCTURE ONLY, like qrita_oracle: nothing on the product path
imports it, and it shares no code with the CUDA library.

Plain fp64 definitions, one row at a time (the row contract is the one
include/qrita.h states):

* ``row_softmax(x, mask, token, inv_t)``: the probabilities over the kept set,
  the token's log-probability and the entropy;
* ``dlogp`` / ``dentropy``: their gradients with respect to the logits;
* ``policy_row``: the clipped policy term with its KL and entropy terms, and
  its derivatives with respect to logp and the entropy;
* ``preference``: sequence sums, pair losses and the weight of every row's
  dlogp.

Pins: tests/test_oracle_losses.py (exact rational probabilities, hand-worked
clip cases, differences of the losses against the gradients, planted
mistakes).
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np


@dataclass
class RowSoftmax:
    p: np.ndarray  # [V], 0 off the kept set
    logp: float
    entropy: float
    ignored: bool

    @property
    def joins(self) -> bool:
        """Whether the row takes part in losses (a NaN does)."""
        return not self.ignored and self.logp != -np.inf


def row_softmax(x, mask, token: int, inv_t: float = 1.0) -> RowSoftmax:
    x = np.asarray(x, dtype=np.float64)
    V = x.shape[0]
    if not 0 <= token < V:
        return RowSoftmax(np.zeros(V), 0.0, 0.0, True)
    kept = np.ones(V, bool) if mask is None else np.asarray(mask) != 0
    p = np.zeros(V)
    xs = x[kept]
    if xs.size == 0 or (np.isneginf(xs)).all():
        return RowSoftmax(p, -np.inf, 0.0, False)
    if np.isnan(xs).any() or np.isposinf(xs).any():
        p[kept] = np.nan
        return RowSoftmax(p, np.nan, np.nan, False)
    y = (xs - xs.max()) * inv_t
    e = np.exp(y)
    s = e.sum()
    p[kept] = e / s
    logs = np.full(V, -np.inf)
    logs[kept] = y - np.log(s)
    pos = p > 0
    return RowSoftmax(p, float(logs[token]), float(-(p[pos] * logs[pos]).sum()), False)


def dlogp(r: RowSoftmax, token: int, inv_t: float) -> np.ndarray:
    """Gradient of logp (0 where the row does not join)."""
    if not r.joins:
        return np.zeros_like(r.p)
    g = -r.p.copy()
    g[token] += 1.0
    return g * inv_t


def dentropy(r: RowSoftmax, inv_t: float) -> np.ndarray:
    if r.ignored:
        return np.zeros_like(r.p)
    g = np.zeros_like(r.p)
    pos = ~(r.p == 0)
    g[pos] = -r.p[pos] * (np.log(r.p[pos]) + r.entropy) * inv_t
    return g


def policy_row(r: RowSoftmax, old, ref, adv, clip_low, clip_high, kl_coef, entropy_coef):
    """(loss, kl, d loss / d logp, d loss / d entropy) of one row."""
    if not r.joins:
        return 0.0, 0.0, 0.0, 0.0
    rho = float(np.exp(r.logp - (r.logp if old is None else old)))
    near = min(max(rho, 1 - clip_low), 1 + clip_high)
    loss = max(-adv * rho, -adv * near)
    binds = (adv > 0 and rho > 1 + clip_high) or (adv < 0 and rho < 1 - clip_low)
    d = 0.0 if binds else -adv * rho
    kl = 0.0
    if ref is not None:
        q = ref - r.logp
        kl = float(np.expm1(q) - q)
        loss += kl_coef * kl
        d += kl_coef * (1 - float(np.exp(q)))
    return loss - entropy_coef * r.entropy, kl, d, -entropy_coef


def softplus(x: float) -> float:
    return float(np.logaddexp(0.0, x))


def preference(rows, starts, ref, weights, beta, label_smoothing=0.0, margin=0.0, length_norm=False):
    """(loss, pair losses, ratios, sequence sums, weight of each row's dlogp)
    from the rows' RowSoftmax."""
    P = len(starts) // 2
    seq, scale = np.zeros(2 * P), np.ones(2 * P)
    for s in range(2 * P):
        vals = [rows[i].logp for i in range(starts[s], starts[s + 1]) if rows[i].joins]
        if length_norm and vals:
            scale[s] = 1.0 / len(vals)
        seq[s] = sum(vals) * scale[s]
    rel = seq - (np.zeros(2 * P) if ref is None else np.asarray(ref, np.float64))
    ratio = rel[0::2] - rel[1::2]
    z = beta * ratio - margin
    pair = np.array([(1 - label_smoothing) * softplus(-v) + (label_smoothing * softplus(v) if label_smoothing else 0.0) for v in z])
    w = np.full(P, 1.0 / P) if weights is None and P else np.asarray(weights if weights is not None else [], np.float64)
    coef = np.zeros(len(rows))
    for i in range(P):
        sig = float(np.exp(-softplus(-z[i])))  # sigmoid
        d = w[i] * beta * (label_smoothing * sig - (1 - label_smoothing) * (1 - sig))
        for s, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
            for j in range(starts[s], starts[s + 1]):
                if rows[j].joins:
                    coef[j] = sign * d * scale[s]
    return float(np.dot(w, pair)) if P else 0.0, pair, ratio, seq, coef
