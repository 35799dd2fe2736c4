"""Cross entropy of a vocabulary head in float64: logits of bf16 hidden states
and a bf16 head, the loss and log-sum-exp of counted rows, and the gradients
of sum_t d_t loss_t with respect to both operands.

A row counts when 0 <= label < vocab.  Everything is formed row by row from
the definition; rows that do not count contribute nothing anywhere.  A row
with a word at +infinity, its label or another, has no loss: NaN.
"""

import numpy as np


def counted(labels, vocab):
    return (labels >= 0) & (labels < vocab)


def head_loss(x, w, labels):
    """(loss, lse) of every row, float64; 0 where a row does not count."""
    rows, vocab = x.shape[0], w.shape[0]
    loss, lse = np.zeros(rows), np.zeros(rows)
    w = w.astype(np.float64)
    for t in np.flatnonzero(counted(labels, vocab)):
        z = w @ x[t].astype(np.float64)
        top = z.max()
        lse[t] = top + np.log(np.exp(z - top).sum())
        others = np.delete(z, labels[t])
        if z[labels[t]] == np.inf:          # an infinity less an infinity
            loss[t] = np.nan
        elif others.size:
            o = others.max()
            if o == -np.inf and z[labels[t]] > o:      # no other word has a share
                continue
            d = (o - z[labels[t]]) + np.log(np.exp(others - o).sum())
            loss[t] = np.log1p(np.exp(d)) if d < 30 else d + np.log1p(np.exp(-d))
    return loss, lse


def head_gradient(x, w, labels, dloss=None):
    """(dx, dw, G) in float64; dloss None: the mean over counted rows."""
    rows, vocab = x.shape[0], w.shape[0]
    on = counted(labels, vocab)
    if dloss is None:
        dloss = np.full(rows, 1.0 / max(1, int(on.sum())))
    w = w.astype(np.float64)
    g = np.zeros((rows, vocab))
    for t in np.flatnonzero(on):
        z = w @ x[t].astype(np.float64)
        p = np.exp(z - z.max())
        p /= p.sum()
        # the label's element without the cancellation of 1 - p
        none = np.isnan(p).any()
        p[labels[t]] = 0.0
        p[labels[t]] = -p.sum() if vocab > 1 else 0.0
        g[t] = dloss[t] * (np.full(vocab, np.nan) if none else p)
    return g @ w, g.T @ x.astype(np.float64), g
