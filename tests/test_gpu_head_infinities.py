"""Logits at infinity in single words of single rows: the loss and the
gradients of every other row are bit for bit what they are without them."""

import pytest
import torch

from bit_nf4_quantized_14_amd import capi
from gpu_util import DEV
from test_gpu_head_loss import make

pytestmark = pytest.mark.gpu

ROW = 5
# the tiles of few rows, of small and of large vocabularies, of many rows, and
# several pieces of the vocabulary
SHAPES = [(20, 64, 300), (20, 72, 17001), (64, 64, 300), (100, 136, 17003), (300, 72, 1500),
          (300, 72, 33000), (20, 8, 530000)]


def run(x, w, lab, dloss):
    f = capi.qn_head_loss_fwd(x, w, lab)
    dx, dw = capi.qn_head_loss_bwd(x, w, lab, f, dloss=dloss, need_dw=True)
    return f, dx, dw


def case(rows, dim, vocab, kind):
    """x, w, labels with column 0 as `kind` needs it, and the value that x[ROW, 0] takes for
    its label's logit to be +infinity."""
    x, w, lab = make(rows, dim, vocab, rows + dim, skip=0.2, lift=0.0)
    word = vocab - 2
    lab[lab == word] = 0
    lab[ROW] = word
    w[:, 0] = 0
    if kind == "weight":             # an infinite element: -infinity to the other rows
        x[:, 0], w[word, 0], value = -1, float("inf"), 1.0
    else:                            # a sum beyond fp32
        x[:, 0], w[word, 0], value = 0, 2.0 ** 70, 2.0 ** 70
    return x.to(DEV), w.to(DEV), lab.to(DEV), value


@pytest.mark.parametrize("kind", ["weight", "overflow"])
@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
def test_a_label_at_infinity_has_no_loss(rows, dim, vocab, kind):
    x, w, lab, value = case(rows, dim, vocab, kind)
    d = torch.rand(rows, device=DEV) + 0.5
    f, dx, _ = run(x, w, lab, d)
    rest = torch.arange(rows, device=DEV) != ROW
    assert torch.isfinite(f.loss[rest]).all() and torch.isfinite(f.lse).all()
    x[ROW, 0] = value
    g, db, dwb = run(x, w, lab, d)
    for t in (g.loss[ROW], g.lse[ROW], g.lse_lo[ROW], g.mean[0], db[ROW], dwb):
        assert torch.isnan(t).all()
    assert g.mean[1] == f.mean[1]
    for a, b in ((g.loss, f.loss), (g.lse, f.lse), (g.lse_lo, f.lse_lo), (db[:, 1:], dx[:, 1:])):
        assert torch.equal(a[rest], b[rest])


def test_one_word_at_infinity():
    x, w = torch.ones(2, 8, device=DEV).bfloat16(), torch.ones(1, 8, device=DEV).bfloat16()
    x[1, 0] = float("inf")
    lab = torch.zeros(2, dtype=torch.int64, device=DEV)
    f, dx, dw = run(x, w, lab, None)
    assert f.loss[0] == 0 and f.lse[0] == 8 and (dx[0] == 0).all()
    for t in (f.loss[1], f.lse[1], f.mean[0], dx[1], dw):
        assert torch.isnan(t).all()


@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
def test_a_label_without_rivals_is_certain(rows, dim, vocab):
    # every other word of one row is at -infinity
    x, w, lab, _ = case(rows, dim, vocab, "overflow")
    w[:, 0] = 2.0 ** 70
    w[lab[ROW], 0] = 0
    d = torch.rand(rows, device=DEV) + 0.5
    f, dx, dw = run(x, w, lab, d)
    rest = torch.arange(rows, device=DEV) != ROW
    x[ROW, 0] = -(2.0 ** 70)
    g, db, dwb = run(x, w, lab, d)
    z = (x[ROW, 1:].double() * w[lab[ROW], 1:].double()).sum()
    slack = (dim + 1) * 2.0 ** -24 * float((x[ROW, 1:].float() * w[lab[ROW], 1:].float()).abs().sum())
    assert g.loss[ROW] == 0 and abs(float(g.lse[ROW]) - float(z)) <= slack + 2.0 ** -24 * abs(float(z))
    assert (db[ROW] == 0).all() and torch.isfinite(dwb).all()
    for a, b in ((g.loss, f.loss), (g.lse, f.lse), (db, dx)):
        assert torch.equal(a[rest], b[rest])
