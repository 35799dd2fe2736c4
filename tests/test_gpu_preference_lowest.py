"""Log-probabilities of rows whose logits are all of their type's lowest (or
another far) value: such a row is uniform, although the log of its sum
vanishes beside the maximum in any one number."""

import numpy as np
import pytest
import torch

from oracle import preference as pr
from bit_nf4_quantized_14_amd import capi

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(2, 1), (2, 7), (3, 100), (2, 9001), (2100, 64),
                                        (2100, 7001)])
def test_rows_of_one_far_value_are_uniform(rows, vocab, dtype):
    """One row split over workgroups, one to a workgroup and one to a wave.
    exp(0) = 1 and the sums of ones are exact, so a token's log-probability is
    -log(vocab) in double and a sequence's is rounded once."""
    f = torch.finfo(dtype)
    for value in (f.min, f.max, 1e30, -1e30):
        x = torch.full((rows, vocab), value, dtype=dtype, device="cuda")
        lab = torch.arange(rows, device="cuda") % vocab
        off = torch.tensor([0, 1, rows], device="cuda")
        logp, lse = capi.qn_seq_logprob(x, lab, off)
        torch.cuda.synchronize()
        want = -np.log(float(vocab)) * np.array([1.0, rows - 1.0])
        got = logp.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= np.abs(want) * U * 1.01), (value, got, want)
        assert bool((lse == x[:, 0].float()).all())


def test_the_oracle_too():
    x = np.full((1, 100), -3.4028234663852886e38)
    logp, _ = pr.seq_logprob(x, np.array([3]), np.array([0, 1]))
    g = pr.seq_logprob_bwd(x, np.array([3]), np.array([0, 1]), np.array([1.0]))
    assert abs(logp[0] + np.log(100)) < 1e-12
    assert abs(g[0, 3] - 0.99) < 1e-12 and abs(g[0, 4] + 0.01) < 1e-12


def test_partly_masked_with_the_lowest_value():
    """Rows in which only some words are left, and a label among the masked
    ones of a row that is masked whole but for -infinity."""
    low = torch.finfo(torch.float32).min
    x = torch.full((4, 500), low, device="cuda")
    x[0, :10] = 2.0                       # ten words left
    x[1, 10:] = float("-inf")             # ten masked words, nothing else
    x[2, :] = float("-inf")
    x[2, 5] = low                         # one masked word
    lab = torch.tensor([3, 4, 5, -1], device="cuda")
    logp, _ = capi.qn_seq_logprob(x, lab, torch.arange(5, device="cuda"))
    want = np.array([-np.log(10), -np.log(10), 0.0, 0.0])
    got = logp.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= np.abs(want) * U * 1.01)
