"""Float64 restatement of the distillation loss, row by row, from its formula.

Shares no code with the GPU path.  ``distill_row`` returns the loss and the
gradient of one row, and the bucket masses a test needs for its bounds.
"""

from __future__ import annotations

import numpy as np


def _lse(x: np.ndarray) -> float:
    m = np.max(x) if x.size else -np.inf
    if not np.isfinite(m):
        return float(m)
    return float(m + np.log(np.sum(np.exp(x - m))))


def distill_row(s, t, idx, temperature=1.0, teacher_lse=None, weight=1.0):
    """s: [V] student logits; t, idx: the teacher's list.  Returns a dict with
    loss, grad [V], q [V], p [V] (the list's mass by column), p_rest, q_rest
    and listed [V]."""
    s = np.asarray(s, np.float64)
    t = np.asarray(t, np.float64)
    idx = np.asarray(idx, np.int64)
    V = s.size
    zero = dict(loss=0.0, grad=np.zeros(V), q=np.zeros(V), p=np.zeros(V), p_rest=0.0, q_rest=1.0,
                listed=np.zeros(V, bool))
    held = (idx >= 0) & (t != -np.inf)
    if weight == 0.0 or not held.any():
        return zero
    if (idx[held] >= V).any():
        return dict(zero, loss=np.nan, grad=np.full(V, np.nan))
    j, u = idx[held], t[held] / temperature
    x = s / temperature
    log_q = x - _lse(x)
    log_p = u - (_lse(u) if teacher_lse is None else float(teacher_lse))
    pk = np.exp(log_p)
    loss = 0.0
    for a in range(j.size):
        if pk[a] > 0:
            loss += pk[a] * (log_p[a] - log_q[j[a]])
    p = np.zeros(V)
    np.add.at(p, j, pk)
    listed = np.zeros(V, bool)
    listed[j] = True
    q = np.exp(log_q)
    p_rest, q_rest, factor = 0.0, 1.0, 1.0
    if teacher_lse is not None and not listed.all():
        p_rest = max(0.0, 1.0 - pk.sum())
        log_q_rest = _lse(log_q[~listed])
        q_rest = np.exp(log_q_rest)
        if p_rest > 0:
            loss += p_rest * (np.log(p_rest) - log_q_rest)
            factor = 1.0 - p_rest / q_rest if q_rest > 0 else 0.0
    grad = np.where(listed, q - p, q * factor) * weight * temperature
    return dict(loss=weight * temperature ** 2 * loss, grad=grad, q=q, p=p, p_rest=p_rest, q_rest=q_rest,
                listed=listed)
