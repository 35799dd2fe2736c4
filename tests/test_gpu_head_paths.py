"""The head's loss at sizes whose tiles go ways that smaller ones do not, on the
GPU against float64 (tests/host/head_paths_check.cpp holds the sizes to them):

* dW in tiles of 256 x 256, and over several pieces of G with more rows than a
  block of G has;
* dX in tiles of 256 x 256 that fill a whole round, with tails after it that are
  dealt in step, or one after another, and in smaller tiles that do (a long
  dimension under few rows).

Bounds as in test_gpu_head_loss.py, row by row.
"""

import pytest
import torch

from bit_nf4_quantized_14_amd import capi
from gpu_util import DEV
from test_gpu_head_loss import H, U, make

pytestmark = pytest.mark.gpu


def check(x, w, lab, dloss, need_dw):
    rows, dim = x.shape
    vocab = w.shape[0]
    xd, wd, ld, d64 = x.to(DEV), w.to(DEV), lab.to(DEV), dloss.double()
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    dx, dw = capi.qn_head_loss_bwd(xd, wd, ld, f, dloss=dloss, need_dw=need_dw)
    wf = wd.double()
    wa, wt = wf.abs(), wf.t().contiguous()
    wat = wa.t().contiguous()
    m = int((ld >= 0).sum())
    rw, bw = (torch.zeros_like(wf), torch.zeros_like(wf)) if need_dw else (None, None)
    for a in range(0, rows, 512):
        s = slice(a, a + 512)
        y, xs = ld[s], xd[s].double()
        on, n, yc = y >= 0, torch.arange(y.shape[0], device=DEV), y.clamp(min=0)
        z = torch.mm(xs, wt)
        top, low = z.amax(1), z.amin(1)
        E = (dim + 1) * U * torch.mm(xs.abs(), wat).amax(1)
        el = 2 * E + U * (3 * (top - low) + 2 * top.abs() + 8) + (96 + vocab / 32) * U \
            + 4 * U * (top.abs() + 20)
        lse = torch.logsumexp(z, 1)
        zero = torch.zeros_like(lse)
        for name, got, ref in (("loss", f.loss, lse - z[n, yc]), ("lse", f.lse, lse)):
            err = (got[s].double() - torch.where(on, ref, zero)).abs()
            assert bool((err <= torch.where(on, el, zero)).all()), (name, a, float(err.max()))
        p = torch.softmax(z, 1) * (d64[s] * on)[:, None]
        p[n, yc] = 0
        keep = p.abs()                              # without the label's element
        p[n, yc] = -p.sum(1)
        full = p.abs()
        eg = (el + 2 * E + 2 * U * lse.abs())[:, None]
        ref = torch.mm(p, wf)
        b = H * torch.mm(keep, wa) + torch.mm(full * (eg + (vocab + 8) * U), wa)
        err = (dx[s].double() - ref).abs()
        assert bool((err <= b * (1 + H) + H * ref.abs() + 1e-30).all()), ("dx", a, float(err.max()))
        assert bool((dx[s][~on] == 0).all())
        if need_dw:
            rw += torch.mm(p.t().contiguous(), xs)
            bw += torch.mm((H * keep + full * (H * (1 + H) + eg + (m + 8) * U)).t().contiguous(),
                           xs.abs())
    if need_dw:
        err = (dw.double() - rw).abs()
        assert bool((err <= bw * (1 + H) + H * rw.abs() + 1e-30).all()), ("dw", float(err.max()))


@pytest.mark.parametrize("rows,dim,vocab,skip,need_dw", [
    (520, 1000, 22001, 0.2, True), (17000, 2048, 20000, 0.1, True), (4700, 4096, 3001, 0.1, False),
    (5300, 4352, 3001, 0.0, False), (5, 70400, 2000, 0.0, True), (100, 40008, 2000, 0.0, False)])
def test_paths_of_large_tiles(rows, dim, vocab, skip, need_dw):
    x, w, lab = make(rows, dim, vocab, rows + vocab, skip=skip)
    check(x, w, lab, torch.rand(rows, device=DEV) + 0.5, need_dw)


@pytest.mark.parametrize("rows,dim,vocab", [(520, 64, 22001), (4400, 264, 3001)])
@pytest.mark.parametrize("counted", [0, 1, 30])
def test_few_rows_of_many_count(rows, dim, vocab, counted):
    # plans are made for all rows, the work is that of the counted ones
    x, w, lab = make(rows, dim, vocab, rows + counted, skip=0.0)
    keep = torch.randperm(rows, generator=torch.Generator().manual_seed(counted))[:counted]
    lab = torch.full_like(lab, -100).index_copy(0, keep, lab[keep])
    check(x, w, lab, torch.rand(rows, device=DEV) + 0.5, True)
