"""The head's loss beside large logits on the GPU against float64.

All logits here are exact in fp32: column 0 adds the same large number to all of
a row's (or to its largest alone), column 1 small multiples of 1 / 8.  What is
left, u = 2^-24 and 2^-8 half a bf16 step, does not grow with the logits:
* an exponential: the difference d of two logits is exact or rounded once, its
  product with log2 e twice (the constant's rounding with it), and the value by
  2 u: (3 |d| + 2) u, and 1 below e^-110;
* loss, and lse with lse_lo: that, 96 + vocab / 32 sums of at most 1, the
  result's rounding (lse_lo's: 2^-48 of lse);
* G: loss's and lse's errors and its own exponential's; it is rounded to bf16
  once, but for the label's element, and summed over the vocabulary; results are
  rounded to bf16.  For dW the row's factor times x is rounded once as well.
"""

import numpy as np
import pytest
import torch

import oracle.head as oh
from bit_nf4_quantized_14_amd import capi
from gpu_util import DEV, f64_host
from test_gpu_head_infinities import SHAPES

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8


def check(x, w, lab, spread):
    """`spread`: how far below its row's largest a logit may be and count."""
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    rows, vocab = x.shape[0], w.shape[0]
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    dx, dw = capi.qn_head_loss_bwd(xd, wd, ld, f, dloss=torch.ones(rows, device=DEV), need_dw=True)
    xn, wn, ln = f64_host(x), f64_host(w), lab.numpy()
    loss, lse = oh.head_loss(xn, wn, ln)
    rx, rw, g = oh.head_gradient(xn, wn, ln, np.ones(rows))
    el = U * (3 * spread + 2 + 96 + vocab / 32)
    err = np.abs(f64_host(f.loss) - loss)
    assert (err <= el + 4 * U * loss).all(), err.max()
    err = np.abs(f64_host(f.lse) + f64_host(f.lse_lo) - lse)
    assert (err <= el + 2.0 ** -46 * np.abs(lse)).all(), err.max()
    rest = np.abs(g)
    keep = rest.copy()
    keep[np.arange(rows), ln] = 0
    eg = 2 * el + U * (3 * spread + 2)
    tiny = 2.0 ** -126 * (np.abs(wn).sum(0).max() + np.abs(xn).sum(0).max())
    bx = keep @ np.abs(wn) * H + rest @ np.abs(wn) * (eg + (vocab + 8) * U)
    err = np.abs(f64_host(dx) - rx)
    assert (err <= bx * (1 + H) + H * np.abs(rx) + tiny).all(), err.max()
    bw = (keep * H + rest * (H * (1 + H) + eg + (rows + 8) * U)).T @ np.abs(xn)
    # A sum of fp32 is finite, in any order, as long as its terms' absolute values (with x
    # and G rounded up) add up to less than the type's largest: 1.99609375 * 2^127 is bf16's.
    # Column 0's terms are up to 1.9921875 * 2^127 in one row alone, so that several rows'
    # sum, and the exact dW with it, may lie beyond it: those elements say nothing.
    fits = (rest.T @ np.abs(xn)) * (1 + 4 * H) < 1.99609375 * 2.0 ** 127
    assert fits[:, 1:].all()
    err = np.abs(np.where(fits, f64_host(dw), 0) - np.where(fits, rw, 0))
    assert (err <= bw * (1 + H) + H * np.abs(rw) + tiny).all(), err.max()


def case(rows, dim, vocab, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(rows, dim)
    w = torch.randn(vocab, dim, generator=g)
    lab = torch.randint(0, vocab, (rows,), generator=g)
    return x, w, lab, g


@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
@pytest.mark.parametrize("power", [10, 16, 20])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_same_added_to_all(rows, dim, vocab, power, sign):
    x, w, lab, g = case(rows, dim, vocab, power)
    x[:, 0], w[:, 0] = sign * 2.0 ** power, 1
    x[:, 1], w[:, 1] = 1, torch.randint(-64, 65, (vocab,), generator=g) / 8.0
    check(x.bfloat16(), w.bfloat16(), lab, 16)


@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
@pytest.mark.parametrize("top", [2.0 ** 28, 1.328125 * 2.0 ** 31, 2.0 ** 40, 1.75 * 2.0 ** 99,
                                 1.9921875 * 2.0 ** 127])
def test_a_few_words_at_the_same_large_logit(rows, dim, vocab, top):
    # every 37th word is at the top, the others half as high; every other row's label is
    # among them
    x, w, lab, g = case(rows, dim, vocab, 5)
    x[:, 0] = top
    w[:, 0] = 0.5
    w[::37, 0] = 1
    lab[::2] = lab[::2] // 37 * 37
    check(x.bfloat16(), w.bfloat16(), lab, 0)


@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
@pytest.mark.parametrize("low", [-(2.0 ** 31), -1.9921875 * 2.0 ** 127])
def test_all_words_far_below_zero(rows, dim, vocab, low):
    x, w, lab, g = case(rows, dim, vocab, 6)
    x[:, 0], w[:, 0] = low, 1
    w[::41, 0] = 0.5
    lab[::2] = lab[::2] // 41 * 41
    check(x.bfloat16(), w.bfloat16(), lab, 0)
