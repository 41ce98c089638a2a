"""Float64 forms of the drafter-training operators: top logits with the row's
log-normaliser, distillation from kept logits, cross entropy of a linear head.
Written from the formulas; NumPy only."""

import numpy as np


def log_sum_exp(z):
    """(maximum, log of the sum of exp(z - maximum)) along the last axis; a row of
    -inf gives (-inf, -inf)."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max(axis=-1)
    safe = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        logsum = np.log(np.exp(z - safe[..., None]).sum(axis=-1))
    return m, logsum


def top_logits(z, k, temperature=1.0):
    """ids, values, lse of rows z [R, V]: descending, lower id first among equals;
    -inf and NaN are no candidates (id -1, value -inf where they run out)."""
    z = np.asarray(z, dtype=np.float64)
    R = z.shape[0]
    ids = np.full((R, k), -1, dtype=np.int32)
    values = np.full((R, k), -np.inf)
    lse = np.empty(R)
    for r in range(R):
        cand = np.nonzero(z[r] > -np.inf)[0]
        order = cand[np.lexsort((cand, -z[r, cand]))][:k]
        ids[r, : len(order)] = order
        values[r, : len(order)] = z[r, order]
        m, logsum = log_sum_exp(z[r] / temperature)
        lse[r] = m + logsum if m > -np.inf else -np.inf
    return ids, values, lse


def distill(z, ids, t, temperature=1.0, teacher_lse=None, row_weight=None):
    """loss [R], grad [R, V], and what tolerances need: p [R, K], scattered p [R, V],
    q [R, V]."""
    z = np.asarray(z, dtype=np.float64)
    t = np.asarray(t, dtype=np.float64) / temperature
    R, V = z.shape
    K = ids.shape[1]
    loss, grad = np.zeros(R), np.zeros((R, V))
    ps, pv, qs = np.zeros((R, K)), np.zeros((R, V)), np.zeros((R, V))
    for r in range(R):
        g = (1.0 if row_weight is None else float(row_weight[r])) / temperature
        m, logsum = log_sum_exp(z[r] / temperature)
        empty_row = np.isneginf(m)
        log_q = np.full(V, -np.inf) if empty_row else z[r] / temperature - m - logsum
        qs[r] = np.exp(log_q)
        slots = [k for k in range(K) if 0 <= ids[r, k] < V and t[r, k] > -np.inf]
        if not slots:
            continue
        # the largest and the logarithm of the sum apart: added, they lose the second
        # where the logits are large
        tm, tl = log_sum_exp(t[r, slots]) if teacher_lse is None else (0.0, float(teacher_lse[r]))
        for k in slots:
            log_p = t[r, k] - tm - tl
            p = np.exp(log_p)
            ps[r, k] = p
            pv[r, ids[r, k]] += p
            if p > 0:
                loss[r] += p * (log_p - log_q[ids[r, k]])
        if not empty_row:
            grad[r] = g * (ps[r].sum() * qs[r] - pv[r])
    return loss, grad, ps, pv, qs


def linear_ce(hidden, weight, labels, grad_loss=None):
    """loss [N], grad_hidden, grad_weight, and (z, dz) for tolerances."""
    h, w = np.asarray(hidden, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    labels = np.asarray(labels)
    N, V = h.shape[0], w.shape[0]
    z = h @ w.T
    m, logsum = log_sum_exp(z)
    used = (labels >= 0) & (labels < V)
    at = np.where(used, labels, 0)
    loss = np.where(used, m + logsum - z[np.arange(N), at], 0.0)
    dz = np.exp(z - (m + logsum)[:, None])
    dz[np.arange(N), at] -= 1.0
    g = np.ones(N) if grad_loss is None else np.asarray(grad_loss, dtype=np.float64)
    dz *= np.where(used, g, 0.0)[:, None]
    return loss, dz @ w, dz.T @ h, z, dz
