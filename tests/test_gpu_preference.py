"""GPU parity of sequence log-probabilities, the paired log-ratio loss and
their gradients against the float64 oracle, under bounds counted from the
roundings of the kernels."""

import numpy as np
import pytest
import torch

import oracle
from oracle import preference as pr
from bit_nf4_quantized_14_amd import capi

from gpu_util import f64_host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _problem(lens, vocab, dtype, pad=0, before=0, behind=0, masked=0.3, seed=0, sigma=3.0):
    """Packed sequences of the given lengths; the logits lie in a wider
    buffer whose other columns hold NaN."""
    rng = np.random.default_rng(seed + 31 * vocab + len(lens))
    rows = before + sum(lens) + behind
    x = (rng.standard_normal((rows, vocab)) * sigma).astype(np.float32)
    labels = rng.integers(0, vocab, rows)
    x[np.arange(rows), labels] += 4
    labels[rng.random(rows) < masked] = -100
    offsets = before + np.concatenate([[0], np.cumsum(lens)])
    buf = torch.full((rows, vocab + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, :vocab] = torch.from_numpy(x).to(dtype).cuda()
    logits = buf[:, :vocab]
    return (logits, torch.from_numpy(labels).cuda(), torch.from_numpy(offsets.astype(np.int64)).cuda(),
            f64_host(logits.contiguous()), labels, offsets)


def _lse_bound(x, lse):
    """Largest error of lse of a row: the terms' exponents carry two
    roundings of at most their size (v - m, times log2 e) and the
    exponential's own (2 u); the additions of a thread, a wave, a workgroup
    and the row's workgroups; the rescalings of the running sum, one for each
    step; the rounding of the result."""
    vocab = x.shape[1]
    steps = -(-vocab // 2048)
    span = np.ptp(np.where(np.isfinite(x), x, 0), axis=1)
    return (2 * span + 4 + (8 + 6) * steps + 60) * U + np.abs(lse) * U


def _check_logprob(prob, logp, lse):
    x, labels, offsets = prob[3:]
    rlogp, rlse = pr.seq_logprob(x, labels, offsets)
    tol = _lse_bound(x, rlse)
    got_lse, got_logp = f64_host(lse), f64_host(logp)
    assert np.all(np.abs(got_lse - rlse) <= tol * (rlse != 0))
    tol_s = np.zeros(len(rlogp))
    for s, t, _ in pr.counted_rows(labels, offsets, x.shape[1]):
        tol_s[s] += tol[t]
    tol_s += np.abs(rlogp) * U
    assert np.all(np.abs(got_logp - rlogp) <= tol_s)
    return rlogp, rlse, tol, tol_s


def _check_grad(prob, dl, d, tol_d, tol_lse, dl_dtype):
    """dl against the gradient for d = d(objective)/d(logp) (float64), of
    which the kernel's fp32 is tol_d off."""
    x, labels, offsets = prob[3:]
    ref = pr.seq_logprob_bwd(x, labels, offsets, d)
    rows = pr.counted_rows(labels, offsets, x.shape[1])
    tol = np.zeros_like(ref)
    for s, t, y in rows:
        p = np.exp(x[t] - x[t].max())
        p /= p.sum()
        hit = np.zeros_like(p)
        hit[y] = 1
        arg = np.abs(np.where(np.isfinite(x[t]), x[t], 0)) + np.abs(x[t]).max()
        # exponent: lse's own error, the difference and its scaling; then the
        # exponential, the product with d and the label's addition
        tol[t] = (np.abs(d[s]) * (p * (tol_lse[t] + 2 * arg * U + 6 * U) + hit * 2 * U) +
                  tol_d[s] * (p + hit))
    got = f64_host(dl)[:, :x.shape[1]]
    if dl_dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8
    tol = tol + 1e-37                  # results below the normal range
    counted = np.zeros(x.shape[0], bool)
    counted[[t for _, t, _ in rows]] = True
    assert not got[~counted].any()
    worst = float(np.max(np.abs(got - ref) / tol)) if got.size else 0.0
    print(f"[pref] gradient at {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0


CASES = [
    # lens, vocab, pad, before, behind
    ([1, 1], 1, 0, 0, 0),
    ([2, 0], 7, 1, 0, 0),
    ([0, 0], 8, 0, 0, 3),
    ([1, 5, 0, 3], 255, 1, 2, 3),
    ([17, 4], 2048, 0, 0, 1),
    ([3, 9], 2049, 7, 1, 0),
    ([40, 3, 20, 31], 5003, 5, 0, 0),
    ([7, 6], 32000, 0, 0, 2),
    ([1, 1], 128256, 0, 0, 0),
    ([1100, 600, 500, 300], 300, 4, 5, 20),     # rows not split
    ([1025, 1026], 2113, 7, 0, 0),              # a wave to a row
    ([2] * 140, 64, 0, 1, 1),                   # more sequences than lanes
    ([0, 1, 0, 0, 2, 0, 1, 0] * 600, 9, 0, 2, 3),   # and than their square
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,vocab,pad,before,behind", CASES)
def test_loss_and_gradient(lens, vocab, pad, before, behind, dtype):
    print(f"[pref] lens={lens[:4]} x{len(lens)} V={vocab} pad={pad} {dtype}", flush=True)
    prob = _problem(lens, vocab, dtype, pad, before, behind)
    logits, lab, off, x, labels, offsets = prob
    S, P = len(lens), len(lens) // 2
    rng = np.random.default_rng(S)
    ref = torch.from_numpy(rng.standard_normal(S).astype(np.float32) * 2).cuda()
    beta, smooth = 0.3, 0.1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    logp0, lse0 = capi.qn_seq_logprob(logits, lab, off, status=status)
    f = capi.qn_pref_loss_fwd(logits, lab, off, ref, beta, smooth, status=status)
    dloss = torch.from_numpy(rng.standard_normal(P).astype(np.float32)).cuda()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(f.logp, logp0) and torch.equal(f.lse, lse0)
    rlogp, rlse, tol_lse, tol_s = _check_logprob(prob, f.logp, f.lse)
    r64 = f64_host(ref)
    loss, dlogp = pr.pref_loss(rlogp, r64, beta, smooth)
    # h moves by beta times both sequences' errors; the loss by at most that,
    # its derivative by a quarter of it; one rounding each
    dh = beta * (tol_s[:P] + tol_s[P:])
    assert np.all(np.abs(f64_host(f.loss) - loss) <= dh + loss * U)
    tol_d = np.concatenate([beta * dh / 4] * 2) + np.abs(dlogp) * U
    assert np.all(np.abs(f64_host(f.dlogp) - dlogp) <= tol_d)
    # the mean loss, in every pair of types; NaN in the buffer's rest
    for out in (torch.float32, torch.bfloat16):
        cols = vocab + pad
        dl = torch.full((x.shape[0], cols), float("nan"), dtype=out, device="cuda")
        capi.qn_pref_loss_bwd(logits, lab, off, f, dlogits=dl)
        assert bool((dl[:, vocab:] == 0).all())
        _check_grad(prob, dl, dlogp / P, tol_d / P + np.abs(dlogp / P) * 2 * U, tol_lse, out)
    # a gradient from above, and the log-probabilities' own
    w64 = f64_host(dloss)
    dl = capi.qn_pref_loss_bwd(logits, lab, off, f, dloss=dloss, dl_dtype=capi.QN_F32)
    both = np.concatenate([w64, w64])
    _check_grad(prob, dl, dlogp * both, tol_d * np.abs(both) + np.abs(dlogp * both) * U, tol_lse,
                torch.float32)
    d = torch.from_numpy(rng.standard_normal(S).astype(np.float32)).cuda()
    dl = capi.qn_seq_logprob_bwd(logits, lab, off, lse0, d, dl_dtype=capi.QN_F32)
    _check_grad(prob, dl, f64_host(d), np.zeros(S), tol_lse, torch.float32)


def test_gradient_matches_differences_of_the_loss():
    """Along a random direction of entries +-1, at step e: the difference
    quotient is off by e^2 / 6 of the third derivative (at most 8 for every
    row's log-sum-exp, times beta, and as much from the loss's own) and by
    the two losses' roundings over 2 e."""
    prob = _problem([3, 2, 2, 4], 40, torch.float32, masked=0.2, seed=4)
    logits, lab, off = prob[:3]
    rows = logits.shape[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    d = (torch.randint(0, 2, logits.shape, device="cuda", generator=g) * 2 - 1).float()
    beta, e = 0.25, 2.0 ** -5
    loss = lambda x: float(capi.qn_pref_loss_fwd(x, lab, off, None, beta).loss.double().mean())  # noqa: E731
    f = capi.qn_pref_loss_fwd(logits, lab, off, None, beta)
    dl = capi.qn_pref_loss_bwd(logits, lab, off, f)
    fd = (loss(logits + e * d) - loss(logits - e * d)) / (2 * e)
    got = float((dl.double() * d.double()).sum())
    # x + e d rounds every logit by at most 16 u; 11 rows of a loss
    noise = 2 * (beta * rows * 40 * 2 * U + 4 * U) / (2 * e)
    print(f"[pref] differences {fd} gradient {got}", flush=True)
    assert abs(fd - got) <= e * e / 6 * (2 * 8 * beta * rows) + noise
    assert abs(got) > 0.02


def test_masked_vocabulary_and_lowest_values():
    """-infinity and the types' lowest finite values in places that are not
    labels: as if those words did not exist."""
    for dtype in (torch.float32, torch.bfloat16):
        low = torch.finfo(dtype).min
        prob = _problem([6, 5], 3001, dtype, masked=0.0, seed=8)
        logits, lab, off, x, labels, offsets = prob
        for fill in (float("-inf"), low):
            y = logits.clone()
            dead = np.arange(3001) % 3 == 1
            dead[labels] = False
            y[:, torch.from_numpy(np.nonzero(dead)[0]).cuda()] = fill
            f = capi.qn_pref_loss_fwd(y, lab, off, None, 0.1)
            dl = capi.qn_pref_loss_bwd(y, lab, off, f, dl_dtype=capi.QN_F32)
            live = ~dead
            lab2 = np.cumsum(live)[labels] - 1
            sub = np.ascontiguousarray(x[:, live])
            rlogp, rlse = pr.seq_logprob(sub, lab2, offsets)
            tol = _lse_bound(x, rlse)
            assert np.all(np.abs(f64_host(f.lse) - rlse) <= tol)
            got = f64_host(dl)
            assert not got[:, dead].any() and np.isfinite(got).all()
            assert np.abs(got[:, live]).sum() > 0
    # a row that is all of the lowest value is uniform
    y = torch.full((2, 100), low, dtype=torch.bfloat16, device="cuda")
    lab = torch.tensor([3, 99], device="cuda")
    logp, lse = capi.qn_seq_logprob(y, lab, torch.tensor([0, 1, 2], device="cuda"))
    # log 100 disappears beside 3.4e38 in the sum that lse is; the row's
    # log-probability is formed from that sum in double
    assert torch.equal(lse.cpu(), torch.full((2,), low))
    assert bool(torch.isfinite(logp).all())


def test_rows_without_a_distribution_are_nan_alone():
    prob = _problem([4, 4, 4, 4], 500, torch.float32, masked=0.0, seed=2)
    logits, lab, off = prob[:3]
    y = logits.clone()
    y[1, 7] = float("nan")
    y[5] = float("-inf")
    y[9, 3] = float("inf")
    f = capi.qn_pref_loss_fwd(y, lab, off, None, 0.1)
    dl = capi.qn_pref_loss_bwd(y, lab, off, f, dloss=torch.ones(2, device="cuda"))
    assert torch.isnan(f.logp).cpu().tolist() == [True, True, True, False]
    assert torch.isnan(f.loss).cpu().tolist() == [True, True]
    assert bool(torch.isnan(dl).any(1).all())         # every pair has a broken row
    # a broken row under a label that does not count is not looked at
    lab2 = lab.clone()
    lab2[[1, 5, 9]] = -100
    f = capi.qn_pref_loss_fwd(y, lab2, off, None, 0.1)
    dl = capi.qn_pref_loss_bwd(y, lab2, off, f)
    assert bool(torch.isfinite(f.loss).all()) and bool(torch.isfinite(dl).all())
    assert not bool(dl[[1, 5, 9]].any())


def test_label_of_no_probability():
    """A label at -infinity: logp -infinity, the loss at its end, and a
    gradient that is finite."""
    prob = _problem([2, 2], 50, torch.float32, masked=0.0, seed=1)
    logits, lab, off = prob[:3]
    y = logits.clone()
    y[0, lab[0]] = float("-inf")
    f = capi.qn_pref_loss_fwd(y, lab, off, None, 0.5)
    dl = capi.qn_pref_loss_bwd(y, lab, off, f)
    assert f.logp.cpu().tolist()[0] == float("-inf")
    assert f.loss.cpu().tolist() == [float("inf")]
    assert f.dlogp.cpu().tolist() == [-0.5, 0.5]
    assert bool(torch.isfinite(dl).all())


def test_all_labels_masked():
    prob = _problem([5, 3], 100, torch.bfloat16, masked=1.1)
    logits, lab, off = prob[:3]
    f = capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1)
    dl = capi.qn_pref_loss_bwd(logits, lab, off, f)
    assert not bool(f.logp.any()) and not bool(f.lse.any()) and not bool(dl.any())
    assert abs(float(f.loss[0]) - np.log(2)) <= np.log(2) * U


def test_no_rows():
    e = torch.empty((0, 10), dtype=torch.bfloat16, device="cuda")
    lab = torch.empty(0, dtype=torch.int64, device="cuda")
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    f = capi.qn_pref_loss_fwd(e, lab, off, None, 0.1)
    assert capi.qn_pref_loss_bwd(e, lab, off, f).shape == (0, 10)
    assert not bool(f.logp.any()) and abs(float(f.loss[0]) - np.log(2)) <= np.log(2) * U


def test_bad_labels_and_offsets_are_reported():
    prob = _problem([4, 4], 64, torch.float32, masked=0.0)
    logits, lab, off = prob[:3]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = lab.clone()
    bad[2] = 64
    bad[5] = 1 << 40
    f = capi.qn_pref_loss_fwd(logits, bad, off, None, 0.1, status=status)
    dl = capi.qn_pref_loss_bwd(logits, bad, off, f)
    masked = bad.clone()
    masked[[2, 5]] = -1
    g = capi.qn_pref_loss_fwd(logits, masked, off, None, 0.1)
    assert int(status.item()) == capi.QN_EINVAL
    assert torch.equal(f.logp, g.logp) and not bool(dl[[2, 5]].any())
    for o in ([0, 4, 9], [-1, 4, 8], [0, 5, 4], [9, 9, 9]):
        status.zero_()
        capi.qn_seq_logprob(logits, lab, torch.tensor(o, device="cuda"), status=status)
        assert int(status.item()) == capi.QN_EINVAL, o
        # the backward stays inside its buffers too
        capi.qn_seq_logprob_bwd(logits, lab, torch.tensor(o, device="cuda"),
                                torch.zeros(8, device="cuda"), torch.ones(2, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("lens,vocab", [([30, 21], 2051), ([1500, 700], 251)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_gradient(dtype, lens, vocab):
    prob = _problem(lens, vocab, dtype, pad=5, behind=2)
    logits, lab, off = prob[:3]
    f = capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1)
    want = capi.qn_pref_loss_bwd(logits, lab, off, f)
    got = capi.qn_pref_loss_bwd(logits, lab, off, f, dlogits=logits)
    assert got.data_ptr() == logits.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("rows", [1, 2])
def test_in_place_gradient_of_a_padded_head(rows):
    """Logits and gradient are the same buffer, the gradient with the
    padding columns; a batch may have one row only."""
    prob = _problem([rows, 0], 1003, torch.bfloat16, pad=5, masked=0.0)
    logits, lab, off = prob[:3]
    f = capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1)
    want = capi.qn_pref_loss_bwd(logits, lab, off, f)
    buf = logits.as_strided((rows, 1008), (1008, 1))
    got = capi.qn_pref_loss_bwd(logits, lab, off, f, dlogits=buf)
    assert got.data_ptr() == logits.data_ptr() and not bool(got[:, 1003:].any())
    assert torch.equal(got[:, :1003], want) and bool(want.any())


def test_odd_pitches_and_guard_bands():
    """Rows that start at any element; what lies between them stays."""
    prob = _problem([5, 4], 999, torch.bfloat16, pad=4)
    logits, lab, off = prob[:3]
    assert logits.stride(0) == 1003
    buf = torch.full((9, 1007), 7.0, dtype=torch.bfloat16, device="cuda")
    f = capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1)
    capi.qn_pref_loss_bwd(logits, lab, off, f, dlogits=buf[:, 3:1003])
    want = capi.qn_pref_loss_bwd(logits, lab, off, f)
    assert torch.equal(buf[:, 3:1002], want) and not bool(buf[:, 1002].any())
    assert bool((buf[:, :3] == 7).all()) and bool((buf[:, 1003:] == 7).all())


def test_far_rows():
    """Rows whose elements lie past 2^31."""
    rows, vocab = 70000, 32768
    y = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (0, 65535, 65537, rows - 1):
        y[t] = torch.randn(vocab, device="cuda", generator=g).bfloat16()
    lab = torch.full((rows,), -100, device="cuda")
    lab[[0, 65535, 65537, rows - 1]] = torch.tensor([5, 6, 7, 8], device="cuda")
    off = torch.tensor([0, 65536, rows], device="cuda")
    f = capi.qn_pref_loss_fwd(y, lab, off, None, 0.1)
    pick = torch.tensor([0, 65535, 65537, rows - 1], device="cuda")
    small = y[pick].contiguous()
    g2 = capi.qn_pref_loss_fwd(small, lab[pick], torch.tensor([0, 2, 4], device="cuda"), None, 0.1)
    # the rows are split differently, so the sums may differ in their order
    assert float((f.logp - g2.logp).abs().max()) <= 1e-4
    dl = capi.qn_pref_loss_bwd(y, lab, off, f, dlogits=y)
    d2 = capi.qn_pref_loss_bwd(small, lab[pick], torch.tensor([0, 2, 4], device="cuda"), g2)
    diff = (dl[pick].float() - d2.float()).abs()
    assert float((diff - d2.float().abs() * 2.0 ** -7).max()) <= 1e-7
    assert not bool(dl[1:65535].any()) and not bool(dl[65538:-1].any())


def test_other_streams_and_two_calls_at_once():
    prob = _problem([30, 21, 8, 50], 4001, torch.bfloat16)
    logits, lab, off = prob[:3]
    f = capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1)
    want = capi.qn_pref_loss_bwd(logits, lab, off, f)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1, stream=s) for s in streams]
    dls = [capi.qn_pref_loss_bwd(logits, lab, off, g, stream=s) for g, s in zip(got, streams)]
    torch.cuda.synchronize()
    for g, dl in zip(got, dls):
        assert torch.equal(g.loss, f.loss) and torch.equal(g.logp, f.logp)
        assert torch.equal(dl, want)


def test_default_stream_by_handle_and_by_object():
    prob = _problem([5, 4], 100, torch.float32)
    logits, lab, off = prob[:3]
    want = capi.qn_seq_logprob(logits, lab, off)
    torch.cuda.synchronize()
    for s in (0, torch.cuda.default_stream(), torch.cuda.Stream().cuda_stream):
        got = capi.qn_seq_logprob(logits, lab, off, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_outputs_that_are_not_given_are_set():
    prob = _problem([5, 4], 100, torch.float32)
    logits, lab, off = prob[:3]
    want = capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1)
    loss = torch.empty(1, device="cuda")
    out = capi.PrefLoss(loss, None, None, None)
    assert capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1, out=out) is out
    assert out.loss is loss and torch.equal(loss, want.loss)
    for name in ("logp", "dlogp", "lse"):
        assert torch.equal(getattr(out, name), getattr(want, name))


def test_graph_replays_follow_new_logits():
    prob = _problem([30, 21], 4001, torch.bfloat16, pad=7)
    logits, lab, off = prob[:3]
    rows = logits.shape[0]
    out = capi.PrefLoss(torch.empty(1, device="cuda"), torch.empty(2, device="cuda"),
                        torch.empty(2, device="cuda"), torch.empty(rows, device="cuda"))
    ws = torch.empty(capi.qn_seq_workspace_bytes(rows, 4001, 2), dtype=torch.uint8, device="cuda")
    dl = torch.empty((rows, 4008), dtype=torch.bfloat16, device="cuda")

    def step():
        capi.qn_pref_loss_fwd(logits, lab, off, None, 0.1, out=out, ws=ws)
        capi.qn_pref_loss_bwd(logits, lab, off, out, dlogits=dl)
    from test_gpu_graphs import _capture, _check_replays
    _check_replays(step, [out.loss, out.logp, out.dlogp, out.lse, dl])
    graph = _capture(step)
    logits.mul_(0.5)
    off.copy_(torch.tensor([0, 17, rows], device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    kept = [t.clone() for t in (out.loss, out.logp, dl)]
    step()
    torch.cuda.synchronize()
    for a, b in zip(kept, (out.loss, out.logp, dl)):
        assert torch.equal(a, b)


def test_refusals_on_the_gpu():
    x = torch.zeros((4, 64), device="cuda")
    lab = torch.zeros(4, dtype=torch.int64, device="cuda")
    off = torch.tensor([0, 2, 4], device="cuda")
    bad = [(x.half(), lab, off), (x.t(), lab[:1].expand(64), off), (x, lab.int(), off),
           (x, lab[:3], off), (x, lab.cpu(), off), (x, lab, off.int()), (x, lab, off[:1]),
           (x[:1].expand(4, 64), lab, off)]
    for args in bad:
        with pytest.raises(capi.QNError):
            capi.qn_seq_logprob(*args)
    with pytest.raises(capi.QNError):
        capi.qn_pref_loss_fwd(x, lab, torch.tensor([0, 1, 2, 4], device="cuda"), None, 0.1)
    with pytest.raises(capi.QNError):
        capi.qn_pref_loss_fwd(x, lab, off, torch.zeros(3, device="cuda"), 0.1)
    f = capi.qn_pref_loss_fwd(x, lab, off, None, 0.1)
    for dl in (torch.empty((4, 63), device="cuda"), torch.empty((3, 64), device="cuda"),
               torch.empty((4, 128), device="cuda")[:, ::2], torch.empty((4, 64)), x.half()):
        with pytest.raises(capi.QNError):
            capi.qn_pref_loss_bwd(x, lab, off, f, dlogits=dl)
