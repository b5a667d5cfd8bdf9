"""Float64 CPU oracle of the verification of drafted tokens, written from the definition: probabilities by
log-softmax, one request at a time. A draw or a test that falls next to a border is told apart by how far the
result is from it, so that every result of the kernel can be checked."""
from __future__ import annotations

import math

import numpy as np


def probabilities(z, t):
    """softmax(z / t) in float64; None for a row that has none (a NaN, +inf, or nothing but -inf)."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max() if z.size else -math.inf
    if not math.isfinite(m):
        return None
    with np.errstate(over="ignore"):
        w = np.exp((z - m) / t)
    return w / w.sum()


def first_largest(z):
    z = np.asarray(z, dtype=np.float64)
    return int(z.argmax()) if math.isfinite(z.max()) else -1


def draw_weights(p, q):
    """What the next token is drawn from: max(p - q, 0), or p where that is nothing (q may be None)."""
    r = p if q is None else np.maximum(p - q, 0.0)
    return r if r.sum() > 0 else p


def accept_ratio(target_row, draft_row, d, t):
    """min(1, p_d / q_d) with draft_row None for a token without probabilities; 0 for what is refused anyway."""
    v = len(target_row)
    if not 0 <= d < v:
        return 0.0
    if t == 0:
        return float(first_largest(target_row) == d)
    p = probabilities(target_row, t)
    if p is None:
        return 0.0
    if draft_row is None:
        return float(p[d])
    q = probabilities(draft_row, t)
    if q is None:
        return 0.0
    return min(1.0, p[d] / q[d]) if q[d] > 0 else float(p[d] > 0)


def request_ref(target, draft, tokens, u, u_draw, t, eps=0.0):
    """What one request may return: a list of (accepted, weights to draw from or the token itself), more than one
    where a test is within a relative `eps` of its border. target [k + 1, v], draft [k, v] or None."""
    found = []
    for i in range(len(tokens) + 1):
        row = target[i]
        if i == len(tokens):
            p = None if t == 0 else probabilities(row, t)
            return found + [(i, first_largest(row) if t == 0 else -1 if p is None else p)]
        d, draft_row = int(tokens[i]), None if draft is None else draft[i]
        a = accept_ratio(row, draft_row, d, t)
        if t == 0:
            if a != 1.0:
                return found + [(i, first_largest(row))]
            continue
        p = probabilities(row, t)
        if p is None:
            return found + [(i, -1)]
        if draft_row is None:
            q = np.zeros(len(row))
            if 0 <= d < len(row):
                q[d] = 1.0
        else:
            q = probabilities(draft_row, t)
        refused = (i, draw_weights(p, q))
        if not (u[i] < a):  # (a NaN refuses)
            if u[i] < a * (1 + eps):
                found.append(refused)
                continue
            return found + [refused]
        if a < 1 and u[i] >= a * (1 - eps):
            found.append(refused)


def draw_error(weights, u, token):
    """How far u is outside of the token's part of the running sum, relative to the whole."""
    if not 0 <= token < len(weights):
        return math.inf
    run = np.cumsum(weights) / weights.sum()
    lo = run[token - 1] if token else 0.0
    return max(lo - u, u - run[token], 0.0)
