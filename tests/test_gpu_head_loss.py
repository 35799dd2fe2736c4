"""Cross entropy of a vocabulary head on the GPU against float64.

Bounds are counted, u = 2^-24 being half an fp32 step and 2^-8 half a bf16
step, relative to the value:
* a logit: fp32 sums of exact products, at most (dim + 1) u sum_k |x w| off (E);
* an exponential: its argument is off by u (|l - top| + |top|) log2 e before
  and 2 u after the multiplication, its value by 2 u: e_exp below;
* loss and lse: 2 E + e_exp + a sum of at most 64 + slices + 32 terms + the
  fp32 result;
* dX: G's elements but the label's are rounded to bf16 once (2^-8), and
  follow lse (E, e_exp, u |lse|); sums of `vocab` products (vocab u at most, of
  sum |G W|); the result is rounded to bf16 once;
* dW: as dX, with the row's factor times x rounded to bf16 once as well.
"""

import numpy as np
import pytest
import torch

import oracle.head as oh
from bit_nf4_quantized_14_amd import capi
from gpu_util import DEV, f64_host

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8


def make(rows, dim, vocab, seed, skip=0.3, lift=4.0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(vocab, dim, generator=g) * (scale / dim ** 0.5)).bfloat16()
    lab = torch.randint(0, vocab, (rows,), generator=g)
    x = torch.randn(rows, dim, generator=g) + lift * w[lab].float()
    drop = torch.rand(rows, generator=g) < skip
    lab = torch.where(drop, -1 - torch.randint(0, 200, (rows,), generator=g), lab)
    return x.bfloat16(), w, lab


def bounds(x, w, lab):
    """Per row: bound of a logit, of a probability (relative), of loss and lse."""
    xa, wa = np.abs(f64_host(x)), np.abs(f64_host(w))
    dim, vocab = xa.shape[1], wa.shape[0]
    z = f64_host(x) @ f64_host(w).T
    top, low = z.max(1), z.min(1)
    E = (dim + 1) * U * (xa @ wa.T).max(1)
    e_exp = U * (3 * (top - low) + 2 * np.abs(top) + 8)
    terms = (96 + vocab / 32) * U
    loss = 2 * E + e_exp + terms + 4 * U * (np.abs(top) + 20)
    return E, loss + 2 * E + e_exp, loss


def check(x, w, lab, dloss=None, need_dw=True, with_lo=True):
    rows, vocab = x.shape[0], w.shape[0]
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    xn, wn, ln = f64_host(x), f64_host(w), lab.numpy()
    on = oh.counted(ln, vocab)
    loss, lse = oh.head_loss(xn, wn, ln)
    _, eg, el = bounds(x, w, lab)
    for name, got, ref in (("loss", f.loss, loss), ("lse", f.lse, lse)):
        err = np.abs(f64_host(got) - ref)
        assert (err <= el)[on].all(), (name, err.max())
        assert (f64_host(got)[~on] == 0).all(), name
    mean = f64_host(f.mean)
    assert mean[1] == on.sum()
    want = loss[on].mean() if on.any() else 0.0
    assert abs(mean[0] - want) <= (el[on].mean() if on.any() else 0) + 2 * U * abs(want)
    if not with_lo:
        f.lse_lo = None
    dl = None if dloss is None else dloss.to(DEV)
    dx, dw = capi.qn_head_loss_bwd(xd, wd, ld, f, dloss=dl, need_dw=need_dw)
    rx, rw, g = oh.head_gradient(xn, wn, ln, None if dloss is None else dloss.double().numpy())
    rest = np.abs(g)
    keep = rest.copy()                                # without the label's element
    keep[np.flatnonzero(on), ln[on]] = 0
    eg = (eg + 2 * U * np.abs(lse))[:, None]
    tiny = 2.0 ** -126 * (np.abs(wn).sum(0).max() + np.abs(xn).sum(0).max())
    bx = (keep * H) @ np.abs(wn) + (rest * (eg + (vocab + 8) * U)) @ np.abs(wn)
    err = np.abs(f64_host(dx) - rx)
    assert (err <= bx * (1 + H) + H * np.abs(rx) + tiny).all(), err.max()
    assert (f64_host(dx)[~on] == 0).all()
    if need_dw:
        m = on.sum()
        bw = (keep * H + rest * (H * (1 + H) + eg + (m + 8) * U)).T @ np.abs(xn)
        err = np.abs(f64_host(dw) - rw)
        assert (err <= bw * (1 + H) + H * np.abs(rw) + tiny).all(), err.max()


SHAPES = [(1, 8, 1), (1, 64, 5), (3, 72, 257), (16, 128, 300), (32, 136, 1000), (33, 128, 1000),
          (64, 200, 513), (127, 64, 128), (129, 64, 4097), (300, 512, 5003), (700, 264, 3001)]


@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
def test_shapes(rows, dim, vocab):
    check(*make(rows, dim, vocab, rows + dim))


@pytest.mark.parametrize("rows,dim,vocab", [(300, 72, 33000), (1030, 64, 16400), (520, 1000, 22001)])
def test_large_tiles(rows, dim, vocab):
    check(*make(rows, dim, vocab, rows), need_dw=vocab < 20000)
