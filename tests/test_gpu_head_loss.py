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


def test_whole_and_last_rounds_of_large_tiles():
    check(*make(1500, 72, 17001, 1))


@pytest.mark.parametrize("rows,dim,vocab", [(16, 72, 17000), (64, 136, 17003), (127, 64, 16500),
                                            (200, 64, 20001), (32, 512, 16384), (100, 512, 16385)])
def test_few_rows_of_many_words(rows, dim, vocab):
    check(*make(rows, dim, vocab, rows), need_dw=rows < 100)


def test_weighted_rows_and_outputs_given():
    x, w, lab = make(150, 96, 2000, 1)
    on = oh.counted(lab.numpy(), 2000)
    dloss = torch.randn(150)
    check(x, w, lab, dloss)
    # what belongs to rows that do not count is not read
    hole = torch.where(torch.from_numpy(on), dloss, torch.tensor(float("nan")))
    check(x, w, lab, hole.where(torch.from_numpy(on), torch.zeros(())))
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    a = capi.qn_head_loss_bwd(xd, wd, ld, f, dloss=dloss.to(DEV), need_dw=True)
    b = capi.qn_head_loss_bwd(xd, wd, ld, f, dloss=hole.to(DEV), need_dw=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # given outputs and workspaces of exactly the asked size, each gradient alone
    nf = capi.qn_head_fwd_workspace_bytes(150, 96, 2000)
    out = capi.HeadLoss(torch.empty(150, device=DEV), None)
    g = capi.qn_head_loss_fwd(xd, wd, ld, out=out, ws=torch.empty(nf, dtype=torch.uint8, device=DEV))
    assert g is out and torch.equal(g.loss, f.loss) and torch.equal(g.mean, f.mean)
    for kw in (dict(need_dx=True, need_dw=False), dict(need_dx=False, need_dw=True)):
        nb = capi.qn_head_bwd_workspace_bytes(150, 96, 2000, **kw)
        c = capi.qn_head_loss_bwd(xd, wd, ld, f, dloss=dloss.to(DEV), **kw,
                                  ws=torch.empty(nb, dtype=torch.uint8, device=DEV))
        for i in range(2):
            assert c[i] is None if not list(kw.values())[i] else torch.equal(c[i], a[i])


def test_without_what_lse_loses():
    check(*make(70, 64, 900, 3), with_lo=False)


@pytest.mark.parametrize("rows", [5, 40, 300])
def test_labels_that_do_not_count(rows):
    x, w, lab = make(rows, 64, 700, rows)
    xd, wd = x.to(DEV), w.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    # none counts
    none = torch.full((rows,), -100, device=DEV)
    f = capi.qn_head_loss_fwd(xd, wd, none, status=status)
    dx, dw = capi.qn_head_loss_bwd(xd, wd, none, f, need_dw=True)
    for t in (f.loss, f.lse, f.mean, dx, dw):
        assert (t == 0).all()
    assert status.item() == 0
    # one above the vocabulary: reported, and not counted
    bad = lab.clone()
    bad[rows // 2] = 700
    f = capi.qn_head_loss_fwd(xd, wd, bad.to(DEV), status=status)
    assert status.item() == capi.QN_EINVAL and f.loss[rows // 2] == 0
    check(x, w, bad)


def test_no_rows():
    w = torch.randn(100, 64, device=DEV).bfloat16()
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    lab = torch.empty(0, dtype=torch.int64, device=DEV)
    f = capi.qn_head_loss_fwd(x, w, lab)
    assert f.loss.shape == (0,) and (f.mean == 0).all()
    dx, dw = capi.qn_head_loss_bwd(x, w, lab, f, need_dw=True)
    assert dx.shape == (0, 64) and (dw == 0).all()


@pytest.mark.parametrize("rows", [20, 100, 300])
def test_a_row_that_is_not_finite_keeps_to_itself(rows):
    x, w, lab = make(rows, 64, 1500, 8, skip=0.0)
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    d = torch.full((rows,), 1.0, device=DEV)
    dx, _ = capi.qn_head_loss_bwd(xd, wd, ld, f, dloss=d)
    for value in (float("nan"), float("inf")):
        xb = xd.clone()
        xb[7, 3] = value
        g = capi.qn_head_loss_fwd(xb, wd, ld)
        db, dw = capi.qn_head_loss_bwd(xb, wd, ld, g, dloss=d, need_dw=True)
        rest = torch.arange(rows, device=DEV) != 7
        assert torch.isnan(g.loss[7]) and torch.isnan(db[7]).all() and torch.isnan(g.mean[0])
        assert torch.equal(g.loss[rest], f.loss[rest]) and torch.equal(db[rest], dx[rest])
        assert torch.isnan(dw).all()


def test_label_out_of_reach():
    # the label's logit overflows to -infinity, the others are ordinary
    x, w, lab = make(40, 64, 300, 4, skip=0.0, lift=0.0)
    x[:, 0], w[:, 0] = 0, 0
    x[5, 0], w[lab[5], 0] = 2.0 ** 70, -(2.0 ** 70)
    lab = torch.where((lab == lab[5]) & (torch.arange(40) != 5), (lab + 1) % 300, lab)
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    assert torch.isposinf(f.loss[5]) and torch.isfinite(f.lse).all()
    dx, _ = capi.qn_head_loss_bwd(xd, wd, ld, f)
    assert torch.isfinite(dx).all() and dx[5].abs().max() > 0


def test_a_certain_label_keeps_its_digits():
    # losses from 1e-9 to 1e-2: relative to themselves as exact as the logits
    rows, dim, vocab = 64, 128, 500
    g = torch.Generator().manual_seed(3)
    w = (torch.randn(vocab, dim, generator=g) / dim ** 0.5).bfloat16()
    lab = torch.randint(0, vocab, (rows,), generator=g)
    x = (torch.linspace(8, 28, rows)[:, None] * w[lab].float()).bfloat16()
    f = capi.qn_head_loss_fwd(x.to(DEV), w.to(DEV), lab.to(DEV))
    loss, _ = oh.head_loss(f64_host(x), f64_host(w), lab.numpy())
    _, _, el = bounds(x, w, lab)
    assert loss.min() < 1e-8
    assert (np.abs(f64_host(f.loss) - loss) <= loss * (np.expm1(el) + 4 * U)).all()
    check(x, w, lab)


def test_large_logits():
    check(*make(60, 64, 800, 5, scale=60.0, lift=0.5))


def reference_gpu(x, w, lab, dloss):
    """The definition in float64 on the GPU, 512 rows at a time: loss, lse, dx,
    dw, and sum |G W|, sum |G| |x| without the label's element."""
    xd, wd = x.to(DEV).double(), w.to(DEV).double()
    wt, wa = wd.t().contiguous(), wd.abs()
    rows, dim = x.shape
    loss, lse = torch.zeros(rows, dtype=torch.float64, device=DEV), torch.zeros(
        rows, dtype=torch.float64, device=DEV)
    dx, ax = torch.zeros_like(xd), torch.zeros_like(xd)
    ld = lab.to(DEV)
    for a in range(0, rows, 512):
        z = torch.mm(xd[a:a + 512], wt)
        y, n = ld[a:a + 512], torch.arange(z.shape[0], device=DEV)
        on = y >= 0
        yc = y.clamp(min=0)
        s = torch.logsumexp(z, 1)
        lse[a:a + 512] = torch.where(on, s, 0)
        loss[a:a + 512] = torch.where(on, s - z[n, yc], 0)
        p = torch.softmax(z, 1)
        p[n, yc] = 0
        p *= (dloss[a:a + 512] * on)[:, None]
        ax[a:a + 512] = torch.mm(p.abs(), wa)
        p[n, yc] = -p.sum(1)
        dx[a:a + 512] = torch.mm(p, wd)
    return loss, lse, dx, ax


@pytest.mark.parametrize("rows,dim,vocab", [(17000, 16, 20000),    # pieces of the vocabulary
                                            (4400, 4096, 700),     # a whole round of dX's tiles
                                            (2000, 2048, 9000)])   # tiles in parts
def test_many_rows(rows, dim, vocab):
    x, w, lab = make(rows, dim, vocab, 2, skip=0.1)
    dloss = torch.rand(rows, device=DEV) + 0.5
    loss, lse, dx, ax = reference_gpu(x, w, lab, dloss.double())
    f = capi.qn_head_loss_fwd(x.to(DEV), w.to(DEV), lab.to(DEV))
    got, _ = capi.qn_head_loss_bwd(x.to(DEV), w.to(DEV), lab.to(DEV), f, dloss=dloss)
    # bounds as in check(), each at its largest over the rows
    z = float((x.float().abs().amax(1) * w.float().abs().sum(1).amax()).max())
    E = (dim + 1) * U * float((x.to(DEV).double().norm(dim=1) * w.to(DEV).double().norm(dim=1).amax()).max())
    del z
    top = float(lse.abs().max())
    el = 2 * E + U * (3 * 60 + 2 * top + 8) + (96 + vocab / 32) * U + 4 * U * (top + 20)
    assert (f.loss.double() - loss).abs().max() <= el and (f.lse.double() - lse).abs().max() <= el
    bx = ax * (H + (el + 2 * E + (vocab + 8) * U) * 2)
    err = (got.double() - dx).abs()
    assert bool((err <= bx * (1 + H) + H * dx.abs() + 1e-30).all()), float(err.max())


@pytest.mark.parametrize("rows", [1, 5, 20])
def test_few_rows_over_pieces_of_the_vocabulary(rows):
    # more words than a piece has: labels in the first piece, in the second, at
    # its edges and in the last word
    dim, vocab = 8, 1040000
    x, w, lab = make(rows, dim, vocab, rows, skip=0.2)
    edge = torch.tensor([vocab - 1, 0, 520191, 520192, vocab - 2])[:rows]
    lab[:len(edge)] = edge
    check(x, w, lab, need_dw=True)


def test_gradient_against_differences():
    # dx and dw along directions of single steps of the inputs' grid; the third
    # derivative of a row's loss along d is at most (2 |w d|_max)^3
    rows, dim, vocab = 6, 16, 50
    g = torch.Generator().manual_seed(11)
    x = (torch.randint(-32, 33, (rows, dim), generator=g) / 16.0).bfloat16()
    w = (torch.randint(-32, 33, (vocab, dim), generator=g) / 32.0).bfloat16()
    lab = torch.randint(0, vocab, (rows,), generator=g)
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    ones = torch.ones(rows, device=DEV)
    dx, dw = capi.qn_head_loss_bwd(xd, wd, ld, f, dloss=ones, need_dw=True)
    _, eg, el = bounds(x, w, lab)
    h = 1 / 32.0
    for which, grad in ((0, dx), (1, dw)):
        d = (torch.randint(0, 2, (x, w)[which].shape, generator=g) * 2 - 1).float() * h
        ends = []
        for s in (1, -1):
            t = [x.float(), w.float()]
            t[which] = t[which] + s * d
            ends.append(f64_host(capi.qn_head_loss_fwd(t[0].bfloat16().to(DEV),
                                                       t[1].bfloat16().to(DEV), ld).loss).sum())
        diff = (ends[0] - ends[1]) / 2
        step = (np.abs(f64_host(w)) @ np.full(dim, h)).max() if which == 0 else \
            (np.abs(f64_host(x)) @ np.full(dim, h)).max()
        third = rows * (2 * step) ** 3 / 6
        want = float((grad.double().cpu() * d.double()).sum())
        slack = float((grad.double().cpu().abs() * d.abs().double()).sum()) * 4 * H
        assert abs(diff - want) <= third + slack + 2 * el.sum(), (which, diff, want)


def test_guard_bands_and_repeatability():
    x, w, lab = make(333, 72, 1111, 21)
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    a = capi.qn_head_loss_bwd(xd, wd, ld, f, need_dw=True)
    nf = capi.qn_head_fwd_workspace_bytes(333, 72, 1111)
    nb = capi.qn_head_bwd_workspace_bytes(333, 72, 1111, True, True)

    def guarded(n, dtype):
        es = torch.empty((), dtype=dtype).element_size()
        raw = torch.full((n * es + 8192,), 0x5A, dtype=torch.uint8, device=DEV)
        return raw, raw[:n * es].view(dtype)
    raws = {k: guarded(n, t) for k, n, t in (
        ("loss", 333, torch.float32), ("lse", 333, torch.float32), ("lo", 333, torch.float32),
        ("mean", 2, torch.float32), ("dx", 333 * 72, torch.bfloat16),
        ("dw", 1111 * 72, torch.bfloat16), ("wf", nf, torch.uint8), ("wb", nb, torch.uint8))}
    v = {k: r[1] for k, r in raws.items()}
    out = capi.HeadLoss(v["loss"], v["lse"], v["mean"], v["lo"])
    capi.qn_head_loss_fwd(xd, wd, ld, out=out, ws=v["wf"])
    capi.qn_head_loss_bwd(xd, wd, ld, out, dx=v["dx"].view(333, 72), dw=v["dw"].view(1111, 72),
                          ws=v["wb"])
    torch.cuda.synchronize()
    for k, (raw, view) in raws.items():
        assert (raw[view.numel() * view.element_size():] == 0x5A).all(), k
    assert torch.equal(v["dx"].view(333, 72), a[0]) and torch.equal(v["dw"].view(1111, 72), a[1])
    assert torch.equal(v["loss"], f.loss) and torch.equal(v["mean"], f.mean)


@pytest.mark.parametrize("rows,dim,vocab", [(3, 64, 500), (100, 64, 500), (300, 128, 33000),
                                            (1100, 64, 17000)])
def test_graph_replays(rows, dim, vocab):
    from test_gpu_graphs import _check_replays
    x, w, lab = make(rows, dim, vocab, 2)
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    out = capi.HeadLoss(*(torch.empty(n, device=DEV) for n in (rows, rows, 2, rows)))
    dx, dw = torch.empty_like(xd), torch.empty_like(wd)
    wf, wb = (torch.empty(n, dtype=torch.uint8, device=DEV) for n in (
        capi.qn_head_fwd_workspace_bytes(rows, dim, vocab),
        capi.qn_head_bwd_workspace_bytes(rows, dim, vocab, True, True)))

    def step():
        capi.qn_head_loss_fwd(xd, wd, ld, out=out, ws=wf)
        capi.qn_head_loss_bwd(xd, wd, ld, out, dx=dx, dw=dw, ws=wb)
    _check_replays(step, [out.loss, out.lse, out.mean, out.lse_lo, dx, dw])


def test_other_streams_and_two_calls_at_once():
    x, w, lab = make(400, 256, 5000, 9)
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    a = capi.qn_head_loss_bwd(xd, wd, ld, f, need_dw=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            g = capi.qn_head_loss_fwd(xd, wd, ld, stream=s)
            got.append((g, capi.qn_head_loss_bwd(xd, wd, ld, g, need_dw=True, stream=s)))
    torch.cuda.synchronize()
    for g, b in got:
        assert torch.equal(g.loss, f.loss) and torch.equal(b[0], a[0]) and torch.equal(b[1], a[1])


def test_batches_as_their_callers_hold_them():
    # hidden states that are a view of a padded batch are taken once they are
    # dense; strided ones, other types and hosts are refused
    x, w, lab = make(40, 64, 300, 1)
    xd, wd, ld = x.to(DEV), w.to(DEV), lab.to(DEV)
    f = capi.qn_head_loss_fwd(xd, wd, ld)
    padded = torch.zeros(4, 12, 64, dtype=torch.bfloat16, device=DEV)
    padded[:, :10] = xd.view(4, 10, 64)
    plab = torch.full((4, 12), -100, device=DEV)
    plab[:, :10] = ld.view(4, 10)
    g = capi.qn_head_loss_fwd(padded.view(48, 64), wd, plab.view(48))
    assert torch.equal(g.loss.view(4, 12)[:, :10].reshape(40), f.loss)
    dx, _ = capi.qn_head_loss_bwd(padded.view(48, 64), wd, plab.view(48), g)
    assert (dx.view(4, 12, 64)[:, 10:] == 0).all()
    for bad in ((xd[::2], wd, ld[::2]), (xd, wd[::2], ld), (xd.float(), wd, ld), (xd, wd, ld.int()),
                (xd, wd, lab), (xd, w, ld), (xd, wd, ld[:39]), (xd[:, :60].contiguous(), wd, ld),
                (xd.view(4, 10, 64), wd, ld)):
        with pytest.raises(capi.QNError):
            capi.qn_head_loss_fwd(*bad)
        with pytest.raises(capi.QNError):
            capi.qn_head_loss_bwd(*bad, f)
    with pytest.raises(capi.QNError):
        capi.qn_head_loss_bwd(xd, wd, ld, capi.HeadLoss(f.loss[:39], f.lse))
    with pytest.raises(capi.QNError):
        capi.qn_head_loss_bwd(xd, wd, ld, f, need_dx=False)


def test_two_graphs_with_one_workspace():
    # replayed in turn on one stream they may share it
    from test_gpu_graphs import _capture, _eager_noise
    cases = [make(60, 128, 700, 1), make(300, 128, 33000, 2)]
    n = max(max(capi.qn_head_fwd_workspace_bytes(c[0].shape[0], 128, c[1].shape[0]),
                capi.qn_head_bwd_workspace_bytes(c[0].shape[0], 128, c[1].shape[0], True, True))
            for c in cases)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    graphs, outs, want = [], [], []
    for c in cases:
        x, w, lab = (t.to(DEV) for t in c)
        rows = x.shape[0]
        out = capi.HeadLoss(*(torch.empty(k, device=DEV) for k in (rows, rows, 2, rows)))
        dx, dw = torch.empty_like(x), torch.empty_like(w)

        def step():
            capi.qn_head_loss_fwd(x, w, lab, out=out, ws=ws)
            capi.qn_head_loss_bwd(x, w, lab, out, dx=dx, dw=dw, ws=ws)
        step()
        torch.cuda.synchronize()
        outs.append((out.loss, out.mean, dx, dw, out, x, w, lab))    # all that the graph uses
        want.append([t.clone() for t in outs[-1][:4]])
        graphs.append(_capture(step))
    for rep in range(4):
        for g, o in zip(graphs, outs):
            for t in o[:4]:
                t.fill_(rep)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, r)), rep
        _eager_noise()
