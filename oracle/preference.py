"""Plain CPU form (float64) of sequence log-probabilities, the paired
log-ratio loss (Rafailov et al., "Direct Preference Optimization", 2023,
equation 7, with label smoothing) and their gradients by the logits."""

from __future__ import annotations

import numpy as np


def _log_softmax(row: np.ndarray) -> np.ndarray:
    m = row.max()
    with np.errstate(invalid="ignore"):
        return (row - m) - np.log(np.exp(row - m).sum())


def counted_rows(labels, offsets, vocab):
    """[(sequence, row, label)] of the rows that count."""
    out = []
    for s in range(len(offsets) - 1):
        for t in range(int(offsets[s]), int(offsets[s + 1])):
            if 0 <= labels[t] < vocab:
                out.append((s, t, int(labels[t])))
    return out


def seq_logprob(logits, labels, offsets):
    """(logp [nseq], lse [rows]); lse 0 where a row does not count."""
    rows, vocab = logits.shape
    logp, lse = np.zeros(len(offsets) - 1), np.zeros(rows)
    with np.errstate(invalid="ignore", divide="ignore"):
        for s, t, y in counted_rows(labels, offsets, vocab):
            x = logits[t].astype(np.float64)
            m = x.max()
            log_sum = np.log(np.exp(x - m).sum())
            lse[t] = m + log_sum
            logp[s] += (x[y] - m) - log_sum     # log_sum vanishes beside a far m
    return logp, lse


def seq_logprob_bwd(logits, labels, offsets, dlogp):
    """Gradient of sum_s dlogp_s logp_s by the logits."""
    rows, vocab = logits.shape
    g = np.zeros((rows, vocab))
    for s, t, y in counted_rows(labels, offsets, vocab):
        g[t] = -dlogp[s] * np.exp(_log_softmax(logits[t].astype(np.float64)))
        g[t, y] += dlogp[s]
    return g


def _softplus(x):
    return np.logaddexp(0.0, x)


def pref_loss(logp, ref, beta, smooth=0.0):
    """(loss [P], dlogp [2P]): chosen sequences first, rejected ones after."""
    logp = np.asarray(logp, np.float64)
    ref = np.zeros_like(logp) if ref is None else np.asarray(ref, np.float64)
    P = len(logp) // 2
    d = logp - ref
    h = beta * (d[:P] - d[P:])
    with np.errstate(over="ignore"):
        loss = (1 - smooth) * _softplus(-h) + smooth * _softplus(h)
        dh = smooth / (1 + np.exp(-h)) - (1 - smooth) / (1 + np.exp(h))
    return loss, np.concatenate([beta * dh, -beta * dh])
