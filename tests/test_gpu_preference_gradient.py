"""Gradients where a row's log-sum-exp in one fp32 number is too little: rows
of a type's lowest value, logits far from zero, and labels that hold nearly all
of the probability.  Bounds are counted from the kernels' roundings and hold no
rounding of lse itself."""

import numpy as np
import pytest
import torch

from oracle import preference as pr
from bit_nf4_quantized_14_amd import capi

from gpu_util import f64_host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _sums(x):
    """Relative error of a row's sum and so of each probability (without the
    exponent's): every term's exponent carries two roundings of at most the
    span and its exponential two; the additions of a thread and of a row's
    threads; one rescaling a step."""
    span = np.ptp(np.where(np.isfinite(x), x, 0), axis=1)
    return (2 * span + 4 + 14 * -(-x.shape[1] // 2048) + 60) * U


def _both(x, lab, off, d, inplace=False):
    """The gradient through qn_seq_logprob and through the loss's forward (whose
    dlogp is replaced), fp32, which must agree."""
    lo = torch.full((x.shape[0],), 7.0, device="cuda")
    logp, lse = capi.qn_seq_logprob(x, lab, off, lse_lo=lo)
    dl = capi.qn_seq_logprob_bwd(x, lab, off, lse, d, dl_dtype=capi.QN_F32, lse_lo=lo)
    f = capi.qn_pref_loss_fwd(x, lab, off, None, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(f.lse, lse) and torch.equal(f.lse_lo, lo) and torch.equal(f.logp, logp)
    f.dlogp = d
    one = torch.ones(d.numel() // 2, device="cuda")
    dl2 = capi.qn_pref_loss_bwd(x, lab, off, f, dloss=one, dl_dtype=capi.QN_F32)
    assert torch.equal(dl, dl2)
    return dl, lse, lo


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(2, 100), (2, 9001), (2100, 64), (2100, 7001)])
def test_rows_of_the_lowest_value(rows, vocab, dtype):
    """Each probability is 1 / vocab: the exponent is the rest of lse, log vocab
    to an fp32 rounding, times log2 e (its rounding and the product's), then the
    exponential (2 u) and the product; the label's is expm1 of it (2 u)."""
    n = float(vocab)
    for value in (torch.finfo(dtype).min, 1e30, -1e9):
        x = torch.full((rows, vocab), value, dtype=dtype, device="cuda")
        lab = torch.arange(rows, device="cuda") % vocab
        off = torch.tensor([0, 1, rows], device="cuda")
        d = torch.tensor([1.0, -0.5], device="cuda")
        dl, lse, lo = _both(x, lab, off, d)
        coef = np.full(rows, -0.5)
        coef[0] = 1.0
        want = np.repeat(-coef[:, None] / n, vocab, 1)
        want[np.arange(rows), lab.cpu().numpy()] += coef
        tol = np.abs(want) * (3 * np.log(n) + 4) * U
        tol[np.arange(rows), lab.cpu().numpy()] = (np.log(n) / n + 4) * U
        assert np.all(np.abs(f64_host(dl) - want) <= tol), value


@pytest.mark.parametrize("dtype,shift", [(torch.float32, 1e4), (torch.float32, -3e5),
                                         (torch.float32, 30.0), (torch.bfloat16, 512.0),
                                         (torch.bfloat16, -4096.0)])
@pytest.mark.parametrize("lens,vocab", [([3, 2], 32000), ([1200, 900], 300), ([1200, 900], 7003)])
def test_logits_far_from_zero(lens, vocab, dtype, shift):
    rng = np.random.default_rng(vocab)
    rows = sum(lens)
    x = (torch.from_numpy(rng.standard_normal((rows, vocab)) * 3) + shift).to(dtype)
    labels = rng.integers(0, vocab, rows)
    labels[rng.random(rows) < 0.2] = -100
    offsets = np.concatenate([[0], np.cumsum(lens)])
    d = np.array([1.0, -0.25])
    dl, lse, lo = _both(x.cuda(), torch.from_numpy(labels).cuda(), torch.from_numpy(offsets).cuda(),
                        torch.tensor(d, dtype=torch.float32, device="cuda"))
    x64 = x.double().numpy()
    ref = pr.seq_logprob_bwd(x64, labels, offsets, d)
    _, rlse = pr.seq_logprob(x64, labels, offsets)
    top = _sums(x64)
    on = labels >= 0
    both = f64_host(lse) + f64_host(lo)
    # the sum's relative error, the rest's own rounding
    assert np.all(np.abs(both - rlse)[on] <= (top + U * U * np.abs(rlse) + 20 * U)[on])
    assert not lo.cpu().numpy()[~on].any()
    coef = np.where(np.arange(rows) < lens[0], d[0], d[1])
    p = np.abs(ref / coef[:, None])
    p[np.arange(rows)[on], labels[on]] = 1 - p[on, labels[on]]
    # exponent: differences of at most t, each rounded (2), the constant and the
    # product (2); exponential and product
    t = np.abs(x64 - rlse[:, None])
    tol = np.abs(coef)[:, None] * p * (top[:, None] + (4 * t + 8) * U)
    # the label's 1 - p moves by p times the exponent's error
    tol[np.arange(rows)[on], labels[on]] += 4 * U * np.abs(ref[on, labels[on]])
    assert np.all((np.abs(f64_host(dl) - ref) <= tol + 1e-37)[on])
    assert not f64_host(dl)[~on].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,team,chunk", [
    (2, 32000, 256, 2048), (2, 700, 256, 2048), (2100, 32000, 256, 32000), (2100, 3000, 64, 3000)])
@pytest.mark.parametrize("above", [20.0, 26.0])
def test_labels_of_nearly_all_the_probability(rows, vocab, team, chunk, above, dtype):
    """All other words `above` below the label's: 1 - p is rest / (1 + rest),
    rest = (vocab - 1) exp(-above).  Up to 16 terms of exp(-20) are below half
    of fp32's step at 1, so the label's thread loses its own words of the rest
    and nothing else; the threads' sums are joined in double."""
    x = torch.full((rows, vocab), 4.0, dtype=dtype, device="cuda")
    lab = torch.arange(rows, device="cuda") * 7919 % vocab
    x[torch.arange(rows, device="cuda"), lab] = 4.0 + above
    off = torch.tensor([0, 1, rows], device="cuda")
    d = torch.tensor([1.0, -0.5], device="cuda")
    dl, _, _ = _both(x, lab, off, d)
    coef = np.full(rows, -0.5)
    coef[0] = 1.0
    rest = (vocab - 1) * np.exp(-above)
    own = 8 * -(-chunk // (8 * team)) / (vocab - 1)
    got = f64_host(dl)
    lab = lab.cpu().numpy()
    hit = got[np.arange(rows), lab] / coef
    err = np.abs(hit / (rest / (1 + rest)) - 1)
    print(f"[pref] 1 - p = {rest / (1 + rest):.4g}, off by {err.max():.2e}", flush=True)
    assert np.all(err <= own + (4 * above + 100) * U)
    got[np.arange(rows), lab] = -coef * np.exp(-above) / (1 + rest)
    p = -got / coef[:, None] * (1 + rest) / np.exp(-above)
    assert np.all(np.abs(p - 1) <= (6 * above + 20) * U)


def test_in_place_and_bf16_gradients_of_confident_labels():
    """In place, the label's logit is read before its gradient is written; a
    bf16 gradient is the fp32 one rounded."""
    rows, vocab = 5, 1003
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((rows, vocab), device="cuda", generator=g).bfloat16()
    lab = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    x[torch.arange(rows, device="cuda"), lab] = 25.0
    off = torch.tensor([0, 3, rows], device="cuda")
    f = capi.qn_pref_loss_fwd(x, lab, off, None, 0.1)
    want = capi.qn_pref_loss_bwd(x, lab, off, f, dl_dtype=capi.QN_F32)
    got = capi.qn_pref_loss_bwd(x, lab, off, f, dlogits=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want.bfloat16())
    assert bool((want[torch.arange(rows, device="cuda"), lab] != 0).all())


def test_lse_lo_of_another_shape_or_type_is_refused():
    x = torch.zeros((4, 64), device="cuda")
    lab = torch.zeros(4, dtype=torch.int64, device="cuda")
    off = torch.tensor([0, 2, 4], device="cuda")
    d = torch.ones(2, device="cuda")
    lse = torch.zeros(4, device="cuda")
    for bad in (torch.zeros(3, device="cuda"), torch.zeros(4, dtype=torch.float64, device="cuda"),
                torch.zeros(4), torch.zeros(8, device="cuda")[::2]):
        with pytest.raises(capi.QNError):
            capi.qn_seq_logprob(x, lab, off, lse_lo=bad)
        with pytest.raises(capi.QNError):
            capi.qn_seq_logprob_bwd(x, lab, off, lse, d, lse_lo=bad)
        f = capi.qn_pref_loss_fwd(x, lab, off, None, 0.1)
        f.lse_lo = bad
        with pytest.raises(capi.QNError):
            capi.qn_pref_loss_bwd(x, lab, off, f)
        with pytest.raises(capi.QNError):
            capi.qn_pref_loss_fwd(x, lab, off, None, 0.1, out=f)
