"""The three bf16 terms in which s G and s T enter the matrix cores, pinned by
problems whose every other step is exact: G, T, A and the restored X pick single
elements, so each gradient is a sum of few fp32 products and two terms (2^-17
of a value lost) miss the bound by far.  dX is compared on both of its paths."""

import numpy as np
import pytest
import torch

import oracle
from oracle import act8 as a8
from oracle import dropout as dr
from bit_nf4_quantized_14_amd import capi

from gpu_util import bf16_dev, f32_dev, f64_host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ALPHA = 1.7


def _problem(m, n, k, r):
    """dY, A and X with one element a row (a column for A), B and T random, the
    weight zero."""
    rng = np.random.default_rng(m + n + k + r)
    dy, x, a = np.zeros((m, n)), np.zeros((m, k)), np.zeros((r, k))
    dy[np.arange(m), np.arange(m) * 5 % n] = 1.0
    x[np.arange(m), np.arange(m) * 7 % k] = np.where(np.arange(m) % 2, 1.0, -1.0)
    a[np.arange(k) % r, np.arange(k)] = np.where(np.arange(k) % 3, 1.0, -1.0)
    b = oracle.bf16_rne_bits(rng.standard_normal((n, r)).astype(np.float32))
    ts = rng.standard_normal((m, r)).astype(np.float32)
    bits = [oracle.bf16_rne_bits(v.astype(np.float32)) for v in (dy, x, a)]
    return bits, b, ts


def _run(m, n, k, r, p=0.0, seed=0, dx_dtype=capi.QN_F32):
    (dy, x, a), b, ts = _problem(m, n, k, r)
    w = capi.nf4_quantize(torch.zeros((n, k), device="cuda"))
    x8 = capi.qn_act8_encode(bf16_dev(x))
    got = capi.qlora_linear_bwd_act8(bf16_dev(dy), x8, w, bf16_dev(a), bf16_dev(b), r, ALPHA,
                                     f32_dev(ts), p=p, seed=seed, dx_dtype=dx_dtype)
    torch.cuda.synchronize()
    f = oracle.bf16_bits_to_f64
    s = float(np.float32(ALPHA) / np.float32(r))
    xr, mask = a8.decode_bf16_bits(*a8.encode(x)), 1.0
    if p > 0:
        xr = dr.dropout_x_bits(xr, p, seed)
        mask = np.where(dr.keep_mask(m, k, p, seed), float(dr.keep_scale(p)), 0.0)
    G, xr, dyf, af = f(dy) @ f(b), f(xr), f(dy), f(a)
    want = (s * (G @ af) * mask, s * (G.T @ xr), s * (dyf.T @ ts.astype(np.float64)))
    # sums of `many` values of one size, each rounded: s times it, its three
    # terms (each addition one; 2^-26 lost), the sum's additions, the mask
    mag = (np.abs(want[0]), s * (np.abs(G).T @ np.abs(xr)), s * (np.abs(dyf).T @ np.abs(ts)))
    many = (1, -(-m // k) + 1, -(-m // n) + 1)
    for name, g, ref, size, c in zip(("dX", "dA", "dB"), got, want, mag, many):
        err = np.abs(f64_host(g) - ref)
        print(f"[terms] M={m} N={n} K={k} r={r} p={p} {name}: "
              f"{float((err / np.maximum(size, 1e-30)).max() / U):.2f} u", flush=True)
        yield name, err, size * (5 + 3 * c) * U, ref


RANKS = [1, 4, 8, 9, 16, 17, 24, 33, 64, 65, 100, 128, 131, 160, 256]


@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("m,n,k", [(1003, 64, 1088), (64, 136, 320), (300, 264, 1024)])
def test_three_terms(m, n, k, r):
    for name, err, tol, _ in _run(m, n, k, r):
        assert np.all(err <= tol), name


@pytest.mark.parametrize("m,n,k,r", [
    (2050, 264, 6208, 16), (2050, 264, 6208, 40),          # 256-wide tiles
    (520, 2112, 2112, 24), (257, 4096, 4160, 12)])         # split tiles
def test_three_terms_in_every_tile(m, n, k, r):
    for name, err, tol, _ in _run(m, n, k, r):
        assert np.all(err <= tol), name


@pytest.mark.parametrize("m,n,k,r", [(1003, 64, 1088, 24), (64, 136, 320, 9),
                                     (2050, 264, 6208, 16)])
def test_three_terms_with_dropout(m, n, k, r):
    for name, err, tol, _ in _run(m, n, k, r, p=0.3, seed=77):
        assert np.all(err <= tol), name


@pytest.mark.parametrize("m,n,k,r", [(1003, 64, 1088, 24), (64, 136, 320, 9)])
def test_a_bf16_dx_is_the_rounded_one(m, n, k, r):
    """One rounding to bf16, of a value that two terms leave within 2^-17."""
    name, err, _, ref = next(_run(m, n, k, r, dx_dtype=capi.QN_BF16))
    assert name == "dX" and np.all(err <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -16))


@pytest.mark.parametrize("m,two", [((1 << 21) - 1, False), (1 << 21, True)])
def test_as_many_tokens_as_a_buffer_resource_spans(m, two):
    """The last number of tokens whose third term fits at r = 256, and the first
    that goes without it: 2^-17 of s G may be lost there."""
    n, k, r = 8, 64, 256
    bf = dict(dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    at = torch.arange(m, device="cuda")
    dy = torch.zeros((m, n), **bf)
    dy[at, at % n] = 1.0
    x = torch.zeros((m, k), **bf)
    x[at, at % k] = 1.0
    a = torch.zeros((r, k), **bf)
    a[torch.arange(k, device="cuda") * 3 + 1, torch.arange(k, device="cuda")] = 1.0
    b = torch.randn((n, r), device="cuda", generator=g).bfloat16()
    ts = torch.ones((m, r), device="cuda")
    w = capi.nf4_quantize(torch.zeros((n, k), device="cuda"))
    x8 = capi.qn_act8_encode(x)
    dx, da, db = capi.qlora_linear_bwd_act8(dy, x8, w, a, b, r, ALPHA, ts)
    torch.cuda.synchronize()
    s = float(np.float32(ALPHA) / np.float32(r))
    sg = s * b.double()                                   # s G of token m: row m % n
    for first in range(0, m, 1 << 18):                    # a quarter million tokens at a time
        rows = at[first:first + (1 << 18)]
        want = sg[rows % n][:, 1:3 * k:3]
        err = (dx[rows].double() - want).abs() / want.abs()
        assert float(err.max()) <= (2.0 ** -17 + 4 * U if two else 8 * U), first
    # sums of `count` equal terms: every addition may lose u of the sum
    count = torch.bincount(at % k, minlength=k).double()
    want = (sg.t()[:, torch.arange(k, device="cuda") % n] * count)
    assert bool(((da.double() - want).abs() <= want.abs() * (m // k) * U).all())
    count = torch.bincount(at % n, minlength=n).double()
    assert bool(((db.double() - s * count[:, None]).abs() <= s * count[:, None] * (m // n) * U).all())
