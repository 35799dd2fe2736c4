"""The log-sum-exps of many rows are off to both sides alike: what all rows of a
sequence are off by adds up over its tokens, and pairs whose answers differ in
length do not lose it in the difference."""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_14_amd import capi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(3000, 4000), (3000, 32000), (2500, 128256), (60, 32000)])
def test_rows_have_no_error_in_common(rows, vocab, dtype):
    """Peaked rows, as a trained head gives them.  A bias of a quarter of fp32's
    step at 1 (2^-25) is allowed for the exponential's own errors; log2 e as one
    fp32 number alone makes 5e-8 to 1e-7 here, and fp32 sums of 500 terms of bf16
    logits 3e-8 more.  The rows' random errors leave at most 2^-24 / sqrt(rows)
    of their mean three times over."""
    g = torch.Generator(device="cuda").manual_seed(vocab + rows)
    x = torch.randn((rows, vocab), device="cuda", generator=g) * 2
    lab = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    x.scatter_add_(1, lab[:, None], 6 + 2 * torch.randn((rows, 1), device="cuda", generator=g))
    x = x.to(dtype)
    off = torch.tensor([0, rows], device="cuda")
    lo = torch.empty(rows, device="cuda")
    logp, lse = capi.qn_seq_logprob(x, lab, off, lse_lo=lo)
    ref = torch.cat([torch.logsumexp(p.double(), 1) for p in x.split(250)])
    err = (lse.double() + lo.double() - ref)
    mean = float(err.mean())
    print(f"[sums] {rows}x{vocab} {dtype}: mean {mean:.2e} std {float(err.std()):.2e}", flush=True)
    assert abs(mean) <= 2.0 ** -25 + 3 * 2.0 ** -24 / np.sqrt(rows)
    want = float((x.gather(1, lab[:, None])[:, 0].double() - ref).sum())
    got = float(logp[0])
    assert abs(got - want) <= rows * (2.0 ** -25 + 3 * 2.0 ** -24 / np.sqrt(rows)) + (
        abs(want) * 2.0 ** -24)


def test_a_pair_of_different_lengths():
    """2000 and 20 tokens: h is beta times what is left of two sums of about
    17000, and the loss follows it; both in double until the end."""
    rows, vocab, beta = 2020, 32000, 0.05
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((rows, vocab), device="cuda", generator=g) * 2
    lab = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    off = torch.tensor([0, 2000, rows], device="cuda")
    tok = torch.log_softmax(x.double(), 1).gather(1, lab[:, None])[:, 0]
    c, r = float(tok[:2000].sum()), float(tok[2000:].sum())
    ref = torch.tensor([round(c), round(r)], dtype=torch.float32, device="cuda")
    f = capi.qn_pref_loss_fwd(x, lab, off, ref, beta)
    h = beta * ((c - round(c)) - (r - round(r)))
    # each token's error as above: a common 2^-25 and a random part
    dh = beta * (2020 * 2.0 ** -25 + 3 * 2.0 ** -24 * np.sqrt(2020))
    want = np.log1p(np.exp(-h))
    assert abs(float(f.loss[0]) - want) <= dh + want * 2.0 ** -24
