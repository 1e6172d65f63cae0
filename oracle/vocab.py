"""Operators on vocabulary rows, in float64 from their definitions (include/eagle.h:
eagle_op_token_logprobs, eagle_op_distill_loss, eagle_op_distill_grad), one row at a time."""
from __future__ import annotations

import numpy as np


def _log_softmax(z, temperature):
    """log q of one row, or None when it has no distribution."""
    y = np.asarray(z, np.float64) / temperature
    if np.isnan(y).any() or (y == np.inf).any() or (y == -np.inf).all():
        return None
    y = y - y.max()
    with np.errstate(divide="ignore"):
        return y - np.log(np.exp(y).sum())


def token_logprobs(z, tok: int, k: int, temperature: float = 1.0):
    """(logprob, entropy, lse, idx [k], val [k]) of one row of logits z [vocab]."""
    z = np.asarray(z, np.float64)
    logq = _log_softmax(z, temperature)
    idx, val = np.full(k, -1, np.int32), np.full(k, -np.inf)
    if logq is None:
        return (0.0 if tok == -1 else np.nan), np.nan, np.nan, idx, np.full(k, np.nan)
    some = np.flatnonzero(z > -np.inf)
    q = np.exp(logq[some])
    order = some[np.lexsort((some, -z[some]))][:k]
    idx[:len(order)], val[:len(order)] = order, logq[order]
    lp = 0.0 if tok == -1 else logq[tok] if 0 <= tok < len(z) else np.nan
    lse = z.max() / temperature - logq.max()
    return lp, -(q * logq[some]).sum(), lse, idx, val


def _teacher(t_idx, t_logp, vocab, tail):
    """(listed tokens, their probabilities, what is left to the others); None when the row is broken."""
    p = {}
    for j, lp in zip(np.asarray(t_idx).tolist(), np.asarray(t_logp, np.float64).tolist()):
        if j < -1 or j >= vocab:
            return None
        if j >= 0 and j not in p:
            p[j] = lp
    idx, lp = np.array(list(p), np.int64), np.array(list(p.values()), np.float64)
    if np.isnan(lp).any() or (lp == np.inf).any() or (tail and (lp > np.log(np.finfo(np.float32).max)).any()):
        return None
    if tail:
        pr = np.exp(lp)
        return (idx, pr, max(0.0, 1.0 - pr.sum())) if pr.sum() <= np.finfo(np.float32).max else None
    if not len(lp) or lp.max() == -np.inf:
        return idx, np.zeros(len(lp)), 0.0
    pr = np.exp(lp - lp.max())
    return idx, pr / pr.sum(), 0.0


def distill(z, t_idx, t_logp, temperature: float = 1.0, tail: bool = True, g: float = 1.0):
    """(loss, stats [4], gradient [vocab] times g) of one row."""
    z = np.asarray(z, np.float64)
    t = _teacher(t_idx, t_logp, len(z), tail)
    logq = _log_softmax(z, temperature)
    stats = np.full(4, np.nan)
    rest = None
    if logq is not None:
        m = z.max()
        shift = -logq.max()     # log sum exp((z - m) / T)
        rest = np.ones(len(z), bool)
        if t is not None:
            rest[t[0]] = False
        with np.errstate(divide="ignore"):
            top = logq[rest].max() if rest.any() else -np.inf
            top = top if top > -1e30 else -np.inf
            log_qt = top + np.log(np.exp(logq[rest] - top).sum()) if top > -np.inf else -np.inf
        if t is not None:
            stats[:] = m, shift, 0.0, 0.0
            if tail:
                stats[2:] = (-np.inf, 0.0) if log_qt == -np.inf else (z[rest].max(), log_qt - top)
    if t is None:
        return np.nan, stats, np.full(len(z), np.nan if g else 0.0)
    idx, p, pt = t
    if not len(idx):
        return 0.0, stats, np.zeros(len(z))
    if logq is None:
        return np.nan, stats, np.full(len(z), np.nan if g else 0.0)
    if log_qt == -np.inf:
        pt = 0.0
    on = p > 0
    loss = (p[on] * (np.log(p[on]) - logq[idx[on]])).sum()
    if pt > 0:
        loss += pt * (np.log(pt) - log_qt)
    d = (p.sum() + pt) * np.exp(logq)
    d[idx] -= p
    if pt > 0:
        d[rest] -= pt * np.exp(logq[rest] - log_qt)
    return loss, stats, d * (g / temperature) if g else np.zeros(len(z))
