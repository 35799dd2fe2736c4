"""Labels whose logit is -infinity, on either side of a pair and on both: what
the header states of logp, the loss, dlogp and the gradients."""

import math

import numpy as np
import pytest
import torch

from bit_nf4_quantized_14_amd import capi

pytestmark = pytest.mark.gpu

INF = float("inf")
BETA = 0.5


def _pair(chosen, rejected, vocab=50, rows=(2, 3)):
    """One pair whose sequences have such a label in their first row, or not,
    and a second pair without any."""
    g = torch.Generator(device="cuda").manual_seed(vocab + rows[0])
    n = rows[0] + rows[1]
    x = torch.randn((2 * n, vocab), device="cuda", generator=g)
    lab = torch.randint(0, vocab, (2 * n,), device="cuda", generator=g)
    off = torch.tensor(np.concatenate([[0], np.cumsum([rows[0], rows[0], rows[1], rows[1]])]),
                       device="cuda")
    first = [0, 2 * rows[0]]            # chosen 0, rejected 0 (sequence 2)
    for on, t in zip((chosen, rejected), first):
        if on:
            x[t, lab[t]] = -INF
    return x, lab, off, first


@pytest.mark.parametrize("vocab,rows", [(50, (2, 3)), (9001, (2, 3)), (300, (600, 500))])
@pytest.mark.parametrize("smooth", [0.0, 0.25])
@pytest.mark.parametrize("chosen,rejected", [(True, False), (False, True), (True, True)])
def test_labels_of_no_probability(chosen, rejected, smooth, vocab, rows):
    x, lab, off, first = _pair(chosen, rejected, vocab, rows)
    f = capi.qn_pref_loss_fwd(x, lab, off, None, BETA, smooth)
    ones = torch.ones(2, device="cuda")
    dl = capi.qn_pref_loss_bwd(x, lab, off, f, dloss=ones)
    torch.cuda.synchronize()
    logp = f.logp.cpu().tolist()
    assert [v == -INF for v in logp] == [chosen, False, rejected, False]
    assert all(math.isfinite(logp[s]) for s in (1, 3))
    # the other pair is as if this one were not there
    assert bool(torch.isfinite(f.loss[1])) and bool(torch.isfinite(f.dlogp[[1, 3]]).all())
    n0, n1 = rows
    other = torch.cat([dl[n0:2 * n0], dl[2 * n0 + n1:]])
    assert bool(torch.isfinite(other).all())
    loss, d = f.loss[0].item(), f.dlogp[[0, 2]].cpu().tolist()
    mine = torch.cat([dl[:n0], dl[2 * n0:2 * n0 + n1]])
    if chosen and rejected:
        assert math.isnan(loss) and all(math.isnan(v) for v in d)
        assert bool(torch.isnan(mine).any(1).all())
        return
    if chosen:
        assert loss == INF
        g = -BETA * (1 - smooth)        # h = -infinity
    else:
        assert loss == (INF if smooth > 0 else 0.0)
        g = BETA * smooth               # h = +infinity
    assert d == [g, -g]
    assert bool(torch.isfinite(mine).all())
    # the row itself: coef at the label, -coef p at the others
    t = first[0] if chosen else first[1]
    coef = d[0] if chosen else d[1]
    p = torch.softmax(x[t].double(), 0)
    want = -coef * p
    want[lab[t]] += coef
    assert dl[t, lab[t]].item() == coef
    # the exponents' roundings (two of at most 12, and the constant's: 4 * 12 u)
    # and the exponentials' (2 u), in the sum and in p itself; the additions of
    # a thread (8) and of the row (14), the product
    tol = (2 * (4 * 12 + 2) + 24) * 2.0 ** -24 * (want.abs() + 1e-30)
    assert bool(((dl[t].double() - want).abs() <= tol).all())


def test_a_broken_row_spoils_its_pair_and_no_other():
    """NaN: the row's own gradient and, through dlogp, its pair's; with a dlogp
    from above the row alone."""
    for value in (float("nan"), INF):
        x, lab, off, _ = _pair(False, False)
        x[1, 7] = value
        f = capi.qn_pref_loss_fwd(x, lab, off, None, BETA)
        dl = capi.qn_pref_loss_bwd(x, lab, off, f)
        mine = torch.tensor([True, True, False, False, True, True, True, False, False, False],
                            device="cuda")
        assert bool(torch.isnan(dl[mine]).any(1).all()) and bool(torch.isfinite(dl[~mine]).all())
        assert torch.isnan(f.loss).cpu().tolist() == [True, False]
        assert torch.isnan(f.dlogp).cpu().tolist() == [True, False, True, False]
        dl = capi.qn_seq_logprob_bwd(x, lab, off, f.lse, torch.ones(4, device="cuda"),
                                     lse_lo=f.lse_lo)
        bad = torch.isnan(dl).any(1).cpu().tolist()
        assert bad == [t == 1 for t in range(10)]
