"""The head's oracle against torch's cross entropy in float64, logits at
infinity among them: a label at +infinity has no loss, one at -infinity an
infinite one."""

import numpy as np
import pytest
import torch

import oracle.head as oh

INF = float("inf")


def both(z, label):
    """(loss, lse, gradient by the logits) of one row of logits by the oracle and by torch:
    x is 1 and w holds the logits themselves."""
    z = np.asarray(z, dtype=np.float64)
    x, lab = np.ones((1, 1)), np.array([label])
    with np.errstate(invalid="ignore", divide="ignore"):
        loss, lse = oh.head_loss(x, z[:, None], lab)
        _, _, g = oh.head_gradient(x, z[:, None], lab)
    t = torch.from_numpy(z)[None].requires_grad_(True)
    out = torch.nn.functional.cross_entropy(t, torch.tensor([label]))
    out.backward()
    ref = (out.item(), torch.logsumexp(t, 1).item(), t.grad[0].numpy())
    return (loss[0], lse[0], g[0]), ref


@pytest.mark.parametrize("z,label", [([0.5, -1.0, 2.0], 1), ([30.0, -20.0, 1.0], 0), ([3.0], 0),
                                     ([1.0, -INF, 2.0], 1), ([1.0, -INF, 2.0], 0)])
def test_finite_losses_and_labels_out_of_reach(z, label):
    got, ref = both(z, label)
    assert got[0] == ref[0] or abs(got[0] - ref[0]) <= 1e-13
    assert abs(got[1] - ref[1]) <= 1e-13 and np.abs(got[2] - ref[2]).max() <= 1e-13


@pytest.mark.parametrize("z,label", [([1.0, INF, 2.0], 1), ([-INF, INF, -INF], 1), ([INF], 0),
                                     ([1.0, INF, 2.0], 0), ([INF, INF], 0)])
def test_a_word_at_infinity_leaves_no_loss(z, label):
    # the loss, an infinity less an infinity, and the gradient: torch's too
    got, ref = both(z, label)
    assert np.isnan(ref[0]) and np.isnan(ref[2]).all()
    assert np.isnan(got[0]) and np.isnan(got[2]).all()


@pytest.mark.parametrize("z,label", [([-INF, 2.0, -INF], 1), ([-INF, -INF, 700.0], 2)])
def test_a_label_without_rivals_is_certain(z, label):
    got, ref = both(z, label)
    assert got[0] == ref[0] == 0 and got[1] == ref[1] == z[label]
    assert (got[2] == 0).all() and (ref[2] == 0).all()
