"""Pins of the preference-loss oracle: closed forms, torch's log-softmax and
autograd in float64, and central differences."""

import math

import numpy as np
import torch

from oracle import preference as pr


def _problem(seed=0, rows=9, vocab=13):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((rows, vocab)) * 3
    labels = rng.integers(0, vocab, rows)
    labels[2] = -100
    offsets = np.array([0, 3, 3, 5, 8])      # an empty sequence, a row behind
    ref = rng.standard_normal(4) * 2
    return logits, labels, offsets, ref


def test_uniform_rows_have_the_closed_form():
    logp, lse = pr.seq_logprob(np.zeros((4, 8)), np.array([0, 7, -1, 3]), np.array([0, 4]))
    assert np.allclose(logp, -3 * math.log(8))
    assert np.allclose(lse, [math.log(8), math.log(8), 0, math.log(8)])


def test_equal_ratios_cost_log_two_and_pull_with_half_beta():
    loss, d = pr.pref_loss([-3.0, -5.0], [-3.0, -5.0], 0.2)
    assert np.allclose(loss, math.log(2)) and np.allclose(d, [-0.1, 0.1])


def test_logprob_and_gradient_match_torch_autograd():
    logits, labels, offsets, ref = _problem()
    x = torch.tensor(logits, requires_grad=True)
    ls = torch.log_softmax(x, 1)
    P, beta, e = 2, 0.3, 0.1
    parts = []
    for s in range(4):
        t = [i for i in range(offsets[s], offsets[s + 1]) if labels[i] >= 0]
        parts.append(sum((ls[i, labels[i]] for i in t), torch.zeros((), dtype=torch.float64)))
    logp = torch.stack(parts)
    d = logp - torch.tensor(ref)
    h = beta * (d[:P] - d[P:])
    loss = -(1 - e) * torch.nn.functional.logsigmoid(h) - e * torch.nn.functional.logsigmoid(-h)
    loss.mean().backward()
    got_logp, _ = pr.seq_logprob(logits, labels, offsets)
    got_loss, dlogp = pr.pref_loss(got_logp, ref, beta, e)
    g = pr.seq_logprob_bwd(logits, labels, offsets, dlogp / P)
    assert np.allclose(got_logp, logp.detach().numpy(), rtol=1e-12)
    assert np.allclose(got_loss, loss.detach().numpy(), rtol=1e-12)
    assert np.allclose(g, x.grad.numpy(), rtol=1e-10, atol=1e-14)
    assert not g[2].any() and not g[8].any()


def test_gradient_matches_central_differences():
    logits, labels, offsets, ref = _problem(3)

    def mean_loss(x):
        return pr.pref_loss(pr.seq_logprob(x, labels, offsets)[0], ref, 0.5, 0.05)[0].mean()
    _, dlogp = pr.pref_loss(pr.seq_logprob(logits, labels, offsets)[0], ref, 0.5, 0.05)
    g = pr.seq_logprob_bwd(logits, labels, offsets, dlogp / 2)
    step = 1e-5
    for t in range(logits.shape[0]):
        for v in range(logits.shape[1]):
            e = np.zeros_like(logits)
            e[t, v] = step
            fd = (mean_loss(logits + e) - mean_loss(logits - e)) / (2 * step)
            assert abs(fd - g[t, v]) < 1e-8
