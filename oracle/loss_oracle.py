"""Plain numpy definitions, in 64 bits, of the training-loss entry points:
row packets of a teacher's logits, the distillation loss that reads them, and
a router's balance loss.  One row, one token, one segment at a time, in the
order of the formulas; nothing is shared with the CUDA path."""

from __future__ import annotations

import math

import numpy as np

F64 = np.float64
NEG = -math.inf


def lse(x) -> float:
    """log sum exp; -inf for an empty (or all -inf) list."""
    x = np.asarray(x, F64)
    if x.size == 0:
        return NEG
    m = np.max(x)
    if np.isnan(m):
        return math.nan
    if m == NEG:
        return NEG
    if m == math.inf:
        return math.nan
    return float(m + np.log(np.sum(np.exp(x - m))))


def logits_topk(x, k: int, tau: float):
    """(values[k], indices[k], counts, tail) of every row of x [rows, vocab]."""
    x = np.asarray(x, F64)
    rows, vocab = x.shape
    values, indices = np.zeros((rows, k)), np.full((rows, k), -1, np.int32)
    counts, tail = np.zeros(rows, np.int32), np.zeros(rows)
    for r in range(rows):
        order = sorted(range(vocab), key=lambda v: (
            not math.isnan(x[r, v]), 0.0 if math.isnan(x[r, v]) else -x[r, v], v))
        keep = sorted(v for v in order[:k] if not x[r, v] == NEG)
        counts[r] = len(keep)
        values[r, :len(keep)] = x[r, keep]
        indices[r, :len(keep)] = keep
        rest = np.ones(vocab, bool)
        rest[keep] = False
        tail[r] = lse(x[r, rest] / tau)
    return values, indices, counts, tail


def distill_row(s, idx, t, tail, tau: float):
    """(loss, stats[6], d loss / d s) of one row; ``tail`` None for none.
    stats = (a, L_off - a / tau, L - a / tau, b, D - b / tau, p_off) with a the
    largest live student logit and b the largest live packet value."""
    s = np.asarray(s, F64)
    idx = np.asarray(idx, np.int64)
    t = np.asarray(t, F64)
    live = s != NEG
    inside = np.zeros(s.size, bool)
    inside[idx] = True
    on, off = inside & live, ~inside & live
    t_of = np.full(s.size, NEG)
    t_of[idx] = t
    a = float(np.max(s[live])) if live.any() else 0.0
    b = float(np.max(t_of[on])) if on.any() else 0.0
    b = 0.0 if b == NEG else b
    x, y = (s - a) / tau, (t_of - b) / tau
    l_off = lse(x[off])
    full = lse(x[live])
    has_tail = tail is not None and off.any()
    rest = tail - b / tau if has_tail else NEG
    d = lse(np.append(y[on], [rest]))
    p_off = 0.0 if d == NEG else math.exp(rest - d)
    stats = (a, l_off, full, b, d, p_off)
    grad = np.zeros(s.size)
    if d == NEG:
        return 0.0, stats, grad
    p = np.zeros(s.size)
    p[on] = np.exp(y[on] - d)
    q = np.zeros(s.size)
    q[live] = np.exp(x[live] - full)
    q_off = math.exp(l_off - full) if off.any() else 0.0
    loss = 0.0
    for v in np.flatnonzero(on):
        if p[v] != 0.0:
            loss += p[v] * ((y[v] - x[v]) - (d - full))
    if p_off != 0.0:
        loss += p_off * ((rest - l_off) - (d - full))
    grad[on] = (q[on] - p[on]) / tau
    if off.any():
        grad[off] = (q_off - p_off) * np.exp(x[off] - l_off) / tau
    return float(loss), stats, grad


def distill(s, indices, values, counts, tail, tau: float, row_grad=None):
    """(loss[rows], stats[rows, 6], grad[rows, vocab])."""
    s = np.asarray(s, F64)
    rows = s.shape[0]
    loss, stats, grad = np.zeros(rows), np.zeros((rows, 6)), np.zeros(s.shape)
    for r in range(rows):
        n = values.shape[1] if counts is None else int(min(max(counts[r], 0), values.shape[1]))
        loss[r], stats[r], g = distill_row(
            s[r], indices[r, :n], values[r, :n], None if tail is None else float(tail[r]), tau)
        w = 1.0 if row_grad is None else float(row_grad[r])
        grad[r] = 0.0 if w == 0.0 else w * g
    return loss, stats, grad


def balance(z, ids, offs, alpha: float, beta: float, mask=None, seg_grad=None):
    """(loss[nseg], counts[nseg, experts], tokens[nseg], grad)."""
    z = np.asarray(z, F64)
    experts, k, nseg = z.shape[1], ids.shape[1], len(offs) - 1
    loss, counts = np.zeros(nseg), np.zeros((nseg, experts), np.int32)
    tokens, grad = np.zeros(nseg, np.int32), np.zeros(z.shape)
    for s in range(nseg):
        part = [t for t in range(offs[s], offs[s + 1]) if mask is None or mask[t]]
        n = tokens[s] = len(part)
        for t in part:
            for e in ids[t]:
                if 0 <= e < experts:
                    counts[s, e] += 1
        if n == 0:
            continue
        f = experts * counts[s].astype(F64) / (k * int(n))
        p, sizes = np.zeros((n, experts)), np.zeros(n)
        for i, t in enumerate(part):
            full = lse(z[t])
            if full != NEG:
                e = np.exp(z[t] - np.max(z[t]))
                p[i] = e / np.sum(e)
                sizes[i] = full
        loss[s] = alpha * float(f @ p.mean(0)) + beta * float(np.mean(sizes ** 2))
        w = 1.0 if seg_grad is None else float(seg_grad[s])
        for i, t in enumerate(part):
            grad[t] = w * p[i] * (alpha * (f - f @ p[i]) + 2 * beta * sizes[i]) / n
    return loss, counts, tokens, grad
