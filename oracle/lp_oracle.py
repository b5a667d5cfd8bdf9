"""Float64 reference of the token log probabilities (NumPy, one row at a time where
it matters), independent of the CUDA library: log probabilities of given labels,
entropies, the largest logits and the gradients, from the definitions

    s = z / T,  lse = log sum_j e^{s_j},  logp = s_y - lse,
    entropy = -sum_j p_j log p_j,
    dz_j = (a (1[j = y] - p_j) - b p_j (log p_j + entropy)) / T.
"""
from __future__ import annotations

import numpy as np


def lp_rows_ref(z, labels=None, *, top_k=0, temperature=1.0, ignore_index=-100):
    """(logp or None, entropy, lse, top_logp or None, top_id or None) of logits z."""
    z = np.asarray(z, dtype=np.float64)
    rows, v = z.shape
    logp, ent, lse = np.zeros(rows), np.zeros(rows), np.zeros(rows)
    top_l = np.full((rows, top_k), -np.inf)
    top_i = np.full((rows, top_k), -1, dtype=np.int64)
    for r in range(rows):
        s = z[r] / temperature
        m = s.max()
        if m == -np.inf:
            lse[r], lp = -np.inf, np.full(v, -np.inf)
        else:
            ld = np.log(np.exp(s - m).sum())
            lse[r] = m + ld
            lp = (s - m) - ld  # not s - lse: beside a large m the sum would lose ld
            p = np.exp(lp)
            ent[r] = -(p[p > 0] * lp[p > 0]).sum()
        order = np.argsort(-z[r], kind="stable")[:top_k]
        for q, j in enumerate(order):
            if z[r, j] > -np.inf:
                top_l[r, q], top_i[r, q] = lp[j], j
        if labels is not None:
            y = labels[r]
            if y == ignore_index or not 0 <= y < v:
                ent[r] = 0.0
            else:
                logp[r] = lp[y]
    return (logp if labels is not None else None, ent, lse, top_l if top_k else None,
            top_i if top_k else None)


def lp_grad_ref(z, labels, grad_logp, grad_entropy, *, temperature=1.0, ignore_index=-100):
    """The gradient in z (labels or either upstream gradient may be None)."""
    z = np.asarray(z, dtype=np.float64)
    rows, v = z.shape
    dz = np.zeros((rows, v))
    for r in range(rows):
        y = None if labels is None else labels[r]
        if y is not None and (y == ignore_index or not 0 <= y < v):
            continue
        s = z[r] / temperature
        m = s.max()
        if m == -np.inf:
            continue
        lp = (s - m) - np.log(np.exp(s - m).sum())
        p = np.exp(lp)
        lp0 = np.where(p > 0, lp, 0.0)
        ent = -(p * lp0).sum()
        if grad_logp is not None and y is not None:
            dz[r] -= grad_logp[r] * p
            dz[r, y] += grad_logp[r]
        if grad_entropy is not None:
            dz[r] -= grad_entropy[r] * p * (lp0 + ent)
    return dz / temperature
