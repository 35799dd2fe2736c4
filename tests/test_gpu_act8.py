"""GPU parity of the 8-bit activation checkpoints and of the linear layer's
backward from one.  Codes, scales and restored values are compared bit for
bit with the oracle; the backward's gradients with float64 under a bound
counted from its roundings."""

import numpy as np
import pytest
import torch

import oracle
from oracle import act8 as a8
from oracle import dropout as dr
from bit_nf4_quantized_14_amd import capi
from bit_nf4_quantized_14_amd import workloads as wl

from gpu_util import bf16_dev, bits_host, f32_dev, f64_host, quantize_dev

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 64), (3, 63), (5, 65), (37, 200), (1, 4096), (130, 129),
          (257, 1031), (64, 8192), (0, 64)]


def _values(rows, cols, seed):
    """Normal rows of very different size, with ties and plain zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 10.0 ** rng.integers(-12, 12, (rows, 1))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    if cols > 1:
        x[:, 1] = x[:, 0] / 2
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_encode_and_decode_bit_exact(rows, cols, dtype):
    x = _values(rows, cols, rows * 7 + cols)
    src = oracle.bf16_rne_bits(x) if dtype == "bf16" else x
    print(f"[act8] {rows}x{cols} {dtype}", flush=True)
    t = capi.qn_act8_encode(bf16_dev(src) if dtype == "bf16" else f32_dev(src))
    yb = capi.qn_act8_decode(t)
    yf = capi.qn_act8_decode(t, dtype=capi.QN_F32)
    torch.cuda.synchronize()
    codes, scale = a8.encode(src)
    assert np.array_equal(t.codes.cpu().numpy(), codes)
    assert np.array_equal(t.scale.cpu().numpy().view(np.uint32), scale.view(np.uint32))
    assert np.array_equal(bits_host(yb), a8.decode_bf16_bits(codes, scale))
    assert np.array_equal(yf.cpu().numpy().view(np.uint32),
                          a8.decode_f32(codes, scale).view(np.uint32))


@pytest.mark.parametrize("cols", [64, 100])
def test_edges_of_the_range(cols):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((12, cols)).astype(np.float32)
    x[0] = 0.0
    x[1] = np.where(np.arange(cols) % 2, 2.0 ** -101, -2.0 ** -101)
    x[2, 0] = 0.0
    x[2] *= 2.0 ** -100
    x[3] *= 1e38
    x[3, 0] = 3.3895314e38
    x[4, 5] = np.inf
    x[5, 6] = -np.inf
    x[6, 7] = np.nan
    x[7] = 2.0 ** -140
    x[8] = -0.0
    x[9, 1:] *= 2.0 ** -130
    for src, dev in ((x, f32_dev(x)), (oracle.bf16_rne_bits(x), None)):
        t = capi.qn_act8_encode(dev if dev is not None else bf16_dev(src))
        y = capi.qn_act8_decode(t, dtype=capi.QN_F32).cpu().numpy()
        codes, scale = a8.encode(src)
        assert np.array_equal(t.codes.cpu().numpy(), codes)
        got = t.scale.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(scale))
        assert np.array_equal(got[~np.isnan(got)], scale[~np.isnan(scale)])
        assert np.array_equal(y, a8.decode_f32(codes, scale), equal_nan=True)


def test_unaligned_bases_and_guard_bands():
    """Row slices of odd width start anywhere; nothing outside is written."""
    rows, cols, k = 19, 101, 3
    x = _values(rows + 2 * k, cols, 9)
    bits = oracle.bf16_rne_bits(x)
    X = bf16_dev(bits)
    codes = torch.full((rows + 2 * k, cols), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((rows + 2 * k, 2), 7.0, dtype=torch.float32, device="cuda")
    t = capi.Act8Tensor(codes[k:-k], scale[k:-k], rows, cols)
    capi.qn_act8_encode(X[k:-k], out=t)
    y = torch.full((rows + 2 * k, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    capi.qn_act8_decode(t, out=y[k:-k])
    torch.cuda.synchronize()
    rc, rs = a8.encode(bits[k:-k])
    assert np.array_equal(t.codes.cpu().numpy(), rc)
    assert np.array_equal(t.scale.cpu().numpy(), rs)
    assert np.array_equal(bits_host(y[k:-k]), a8.decode_bf16_bits(rc, rs))
    for part, fill in ((codes, 77), (scale, 7.0), (y, 7.0)):
        assert bool((part[:k] == fill).all()) and bool((part[-k:] == fill).all())


def _bwd_problem(m, n, k, r, seed=0):
    wk = wl.workload("tiny")
    w = wl.weight(wk, 0, rows=n, cols=k)
    x = wl.activations(wk, 0, m=m, k=k)
    a = wl.lora_a(wk, 0, r=r, k=k)
    rng = np.random.default_rng(900 + m + n + seed)
    b = oracle.bf16_rne_bits((rng.standard_normal((n, r)) * 0.3).astype(np.float32))
    return w, x, a, b, wl.grad_out(wk, 0, m=m, n=n)


def _f64(bits):
    return oracle.bf16_bits_to_f64(bits)


def _check_bwd(m, n, k, r, alpha, p=0.0, seed=0, dx_dtype=capi.QN_F32, need_dx=True):
    print(f"[act8 bwd] M={m} N={n} K={k} r={r} p={p} dx={need_dx}", flush=True)
    w, x, a, b, dy = _bwd_problem(m, n, k, r)
    t, _ = quantize_dev(w)
    X, A, B, DY = bf16_dev(x), bf16_dev(a), bf16_dev(b), bf16_dev(dy)
    if p > 0:
        _, ts = capi.qlora_linear_fwd_dropout(X, t, A, B, r, alpha, p, seed)
    else:
        _, ts = capi.qlora_linear_fwd(X, t, A, B, r, alpha)
    x8 = capi.qn_act8_encode(X)
    dx, da, db = capi.qlora_linear_bwd_act8(DY, x8, t, A, B, r, alpha, ts, p=p, seed=seed,
                                            dx_dtype=dx_dtype, need_dx=need_dx)
    torch.cuda.synchronize()
    codes, scale = a8.encode(x)
    xr = a8.decode_bf16_bits(codes, scale)
    rp, rq, rd = oracle.nf4_quantize(w)
    W = _f64(oracle.nf4_dequantize(rp, rq, rd, w.size).reshape(w.shape))
    Af, Bf, DYf, T = _f64(a), _f64(b), _f64(dy), ts.double().cpu().numpy()
    mask = np.ones((m, k))
    Xr = _f64(xr)
    if p > 0:
        Xr = _f64(dr.dropout_x_bits(xr, p, seed))
        mask = np.where(dr.keep_mask(m, k, p, seed), float(dr.keep_scale(p)), 0.0)
    s = float(np.float32(alpha) / np.float32(r))
    G = DYf @ Bf
    aG = np.abs(DYf) @ np.abs(Bf)
    u = 2.0 ** -24
    # every product of two bf16 is exact in fp32; a sum of n of them in any
    # order is off by n u of the sum of magnitudes.  G and T enter the matrix
    # cores as two bf16 (2^-17 of the value at most are lost), after s G and
    # s T were rounded to fp32.
    eG = aG * (n + 2) * u
    res = {}
    ref = s * (G.T @ Xr)
    tol = s * ((eG + np.abs(G) * 2.0 ** -17).T @ np.abs(Xr) + (m + 8) * u * (aG.T @ np.abs(Xr)))
    res["dA"] = (f64_host(da), ref, tol)
    ref = s * (DYf.T @ T)
    mag = np.abs(DYf).T @ np.abs(T)
    res["dB"] = (f64_host(db), ref, s * mag * (2.0 ** -17 + (m + 8) * u))
    if need_dx:
        ref = DYf @ W + s * (G @ Af) * mask
        tol = ((np.abs(DYf) @ np.abs(W)) * (n + 2 * r + 8) * u +
               s * ((eG + aG * (2.0 ** -17 + (n + 2 * r + 8) * u)) @ np.abs(Af)) * mask)
        if dx_dtype == capi.QN_BF16:
            tol = tol * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8
        res["dX"] = (f64_host(dx), ref, tol)
    else:
        assert dx is None
    for name, (got, ref, tol) in res.items():
        worst = float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)))
        print(f"[act8 bwd] {name}: {worst:.3f} of its bound", flush=True)
        assert worst <= 1.0, name
    return DY, x8, t, A, B, ts, (dx, da, db)


@pytest.mark.parametrize("m,n,k,r,alpha", [
    (1, 8, 64, 1, 1.0), (37, 200, 192, 5, 7.0), (16, 64, 4160, 33, 64.0),
    (130, 136, 320, 64, 16.0), (64, 128, 256, 256, 512.0), (300, 264, 1024, 16, 32.0),
    (257, 1024, 576, 16, 32.0), (520, 256, 640, 100, 100.0), (1003, 64, 128, 8, 16.0),
    # few tokens: one, two and four tiles of 16, a half block of columns, one
    # and many slices of the weight's rows; and the first M of the GEMM
    (16, 4096, 1088, 16, 32.0), (17, 1032, 192, 12, 12.0), (33, 1032, 1216, 12, 24.0),
    (64, 520, 4160, 40, 40.0), (65, 520, 320, 16, 16.0),
    # ranks in two parts, and row slices of each width of workgroup
    (200, 136, 192, 160, 160.0), (1500, 72, 64, 200, 200.0), (2100, 64, 64, 64, 64.0),
    (2100, 136, 64, 16, 16.0), (2100, 64, 128, 24, 24.0),
    # B's rows one rank at a time, and whole, for each width of the rank
    (70, 72, 64, 19, 19.0), (70, 72, 64, 131, 131.0), (70, 72, 64, 128, 128.0),
    (70, 72, 64, 37, 37.0), (70, 72, 64, 256, 256.0),
    # several blocks of 64 tokens; the GEMM with 128- and with 256-wide tiles
    (100, 4104, 192, 8, 8.0), (1003, 64, 1024, 8, 16.0), (257, 1024, 2112, 16, 32.0),
    (2050, 264, 6208, 16, 16.0),
])
def test_backward_from_a_checkpoint(m, n, k, r, alpha):
    _check_bwd(m, n, k, r, alpha)


@pytest.mark.parametrize("m,n,k,r,p", [
    (1, 8, 64, 1, 0.5), (37, 200, 192, 5, 0.1), (130, 136, 320, 64, 0.3),
    (64, 128, 256, 256, 0.1), (258, 264, 576, 16, 0.05), (33, 1032, 192, 12, 0.2),
    (700, 72, 64, 160, 0.1), (1100, 64, 64, 24, 0.3), (257, 136, 2112, 16, 0.1),
])
def test_backward_with_dropout(m, n, k, r, p):
    _check_bwd(m, n, k, r, 2.0 * r, p=p, seed=(m * 1000003 + k) | (1 << 40))


@pytest.mark.parametrize("m,n,k,r", [(37, 200, 192, 5), (300, 264, 1024, 16)])
def test_without_dx_the_adapters_get_the_same_gradients(m, n, k, r):
    DY, x8, t, A, B, ts, (_, da, db) = _check_bwd(m, n, k, r, 16.0, dx_dtype=capi.QN_BF16)
    none, da2, db2 = capi.qlora_linear_bwd_act8(DY, x8, t, A, B, r, 16.0, ts, need_dx=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(da, da2) and torch.equal(db, db2)


def test_dx_and_db_do_not_depend_on_the_checkpoint():
    """Given T, X enters dA alone: another checkpoint leaves the bits of dX
    and dB.  Beside qlora_linear_bwd both are within rounding: two results
    within the bounds of _check_bwd of one value (2^-17 of sums of magnitudes
    that here are below 64 times the largest result) differ by twice that."""
    m, n, k, r = 300, 264, 1024, 16
    DY, x8, t, A, B, ts, (dx, da, db) = _check_bwd(m, n, k, r, 32.0)
    other = capi.qn_act8_encode(torch.ones((m, k), dtype=torch.bfloat16, device="cuda"))
    dx1, da1, db1 = capi.qlora_linear_bwd_act8(DY, other, t, A, B, r, 32.0, ts)
    X = bf16_dev(_bwd_problem(m, n, k, r)[1])
    dx0, _, db0 = capi.qlora_linear_bwd(DY, X, t, A, B, r, 32.0, ts)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx1) and torch.equal(db, db1) and not torch.equal(da, da1)
    for u, v in ((dx, dx0), (db, db0)):
        assert float((u - v).abs().max()) <= 2 * 64 * 2.0 ** -17 * float(v.abs().max())


@pytest.mark.parametrize("m,n,k,r", [(40, 72, 128, 8), (200, 264, 1088, 24)])
def test_gradients_match_differences_of_the_forward(m, n, k, r):
    """The layer's output Y is linear in X, in A and in B, each with the others
    held: its difference quotient along a direction D is Y's value there, for
    any step.  So sum(dY * Y_D) must be sum(gradient * D), here for the
    restored X.  Each side is off by at most (n + k + 2 r + m) 2^-24, and
    2^-16 for two splits into two bf16 terms, of the same sum with every
    factor's magnitude."""
    w, x, a, b, dy = _bwd_problem(m, n, k, r)
    t, _ = quantize_dev(w)
    A, B, DY, alpha = bf16_dev(a), bf16_dev(b), bf16_dev(dy), 2.0 * r
    x8 = capi.qn_act8_encode(bf16_dev(x))
    X = capi.qn_act8_decode(x8)
    _, ts = capi.qlora_linear_fwd(X, t, A, B, r, alpha)
    dx, da, db = capi.qlora_linear_bwd_act8(DY, x8, t, A, B, r, alpha, ts)
    g = torch.Generator(device="cuda").manual_seed(2)
    zero = capi.nf4_quantize(torch.zeros((n, k), device="cuda"))
    W = capi.nf4_dequantize(t)

    def direction(like):
        return torch.randn(like.shape, device="cuda", generator=g).bfloat16()
    up = lambda v: v.double()  # noqa: E731
    ab = lambda v: v.double().abs()  # noqa: E731
    for name, grad, d in (("dX", dx, direction(X)), ("dA", da, direction(A)),
                          ("dB", db, direction(B)), ("dX", dx, dx.bfloat16()),
                          ("dA", da, da.bfloat16()), ("dB", db, db.bfloat16())):
        base = t if name == "dX" else zero       # the base product has no part in dA, dB
        x1, a1, b1 = (d if name == "dX" else X, d if name == "dA" else A,
                      d if name == "dB" else B)
        y, _ = capi.qlora_linear_fwd(x1, base, a1, b1, r, alpha)
        one, two = float((up(DY) * up(y)).sum()), float((up(grad) * up(d)).sum())
        mag = 2.0 * ab(x1) @ ab(a1).t() @ ab(b1).t()
        if name == "dX":
            mag = mag + ab(x1) @ ab(W).t()
        bound = float((ab(DY) * mag).sum()) * 2 * ((n + k + 2 * r + m) * 2.0 ** -24 + 2.0 ** -16)
        print(f"[act8 bwd] {name}: {one:.6g} {two:.6g} bound {bound:.3g}", flush=True)
        assert abs(one - two) <= bound


@pytest.mark.parametrize("r", [24, 64, 128, 160])
def test_b_at_any_alignment(r):
    m, n, k = 40, 72, 128
    w, x, a, b, dy = _bwd_problem(m, n, k, r)
    t, _ = quantize_dev(w)
    X, A, B, DY = bf16_dev(x), bf16_dev(a), bf16_dev(b), bf16_dev(dy)
    _, ts = capi.qlora_linear_fwd(X, t, A, B, r, 16.0)
    x8 = capi.qn_act8_encode(X)
    want = capi.qlora_linear_bwd_act8(DY, x8, t, A, B, r, 16.0, ts)
    buf = torch.empty(n * r + 1, dtype=torch.bfloat16, device="cuda")
    B2 = buf[1:].view(n, r)
    B2.copy_(B)
    got = capi.qlora_linear_bwd_act8(DY, x8, t, A, B2, r, 16.0, ts)
    torch.cuda.synchronize()
    for u, v in zip(want, got):
        assert torch.equal(u, v)


def test_a_broken_block_shows_in_da():
    """An infinity in X leaves NaN in the dA columns of its block alone."""
    m, n, k, r = 40, 64, 256, 4
    w, x, a, b, dy = _bwd_problem(m, n, k, r)
    x = x.copy()
    x[7, 70] = 0x7F80
    t, _ = quantize_dev(w)
    x8 = capi.qn_act8_encode(bf16_dev(x))
    ts = torch.zeros((m, r), dtype=torch.float32, device="cuda")
    dx, da, db = capi.qlora_linear_bwd_act8(bf16_dev(dy), x8, t, bf16_dev(a), bf16_dev(b), r,
                                            8.0, ts)
    torch.cuda.synchronize()
    bad = torch.isnan(da).cpu().numpy()
    assert bad[:, 64:128].all() and not bad[:, :64].any() and not bad[:, 128:].any()
    assert bool(torch.isfinite(dx).all()) and bool((db == 0).all())


def test_on_another_stream_and_twice_at_once():
    m, n, k, r = 130, 136, 320, 8
    DY, x8, t, A, B, ts, ref = _check_bwd(m, n, k, r, 16.0)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a = capi.qlora_linear_bwd_act8(DY, x8, t, A, B, r, 16.0, ts, stream=s1)
    b = capi.qlora_linear_bwd_act8(DY, x8, t, A, B, r, 16.0, ts, stream=s2)
    c = capi.qn_act8_decode(x8, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    for u, v, w in zip(ref, a, b):
        assert torch.equal(u, v) and torch.equal(u, w)
    assert torch.equal(c, capi.qn_act8_decode(x8))


def test_graph_of_encode_backward_replays():
    m, n, k, r = 300, 264, 512, 16
    w, x, a, b, dy = _bwd_problem(m, n, k, r)
    t, _ = quantize_dev(w)
    X, A, B, DY = bf16_dev(x), bf16_dev(a), bf16_dev(b), bf16_dev(dy)
    _, ts = capi.qlora_linear_fwd(X, t, A, B, r, 32.0)
    x8 = capi.Act8Tensor.empty(m, k)
    dx = torch.empty((m, k), dtype=torch.bfloat16, device="cuda")
    da = torch.empty((r, k), dtype=torch.float32, device="cuda")
    db = torch.empty((n, r), dtype=torch.float32, device="cuda")
    ws = torch.empty(capi.qlora_bwd_act8_workspace_bytes(m, n, k, r), dtype=torch.uint8,
                     device="cuda")

    def step():
        capi.qn_act8_encode(X, out=x8)
        capi.qlora_linear_bwd_act8(DY, x8, t, A, B, r, 32.0, ts, dx=dx, dA=da, dB=db, ws=ws)
    from test_gpu_graphs import _check_replays
    _check_replays(step, [x8.codes, x8.scale, dx, da, db])


def test_refusals_on_the_gpu():
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (x.half(), x.t(), x[:, ::2], x[0]):
        with pytest.raises(capi.QNError):
            capi.qn_act8_encode(bad)
    t = capi.qn_act8_encode(x)
    with pytest.raises(capi.QNError):
        capi.qn_act8_decode(t, out=torch.empty((4, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(capi.QNError):
        capi.qn_act8_encode(x, out=capi.Act8Tensor.empty(4, 64))
    with pytest.raises(capi.QNError):
        capi.qn_act8_decode(t, dtype=5)


def test_a_weight_elsewhere_or_too_small_is_refused():
    m, n, k, r = 4, 64, 128, 8
    bf = dict(dtype=torch.bfloat16, device="cuda")
    t = capi.qn_act8_encode(torch.ones((m, k), **bf))
    dy, A, B = torch.ones((m, n), **bf), torch.ones((r, k), **bf), torch.ones((n, r), **bf)
    ts = torch.ones((m, r), device="cuda")
    w = capi.nf4_quantize(torch.ones((n, k), device="cuda"))
    host, small = capi.NF4Tensor.empty(n, k, device="cpu"), capi.NF4Tensor.empty(n // 2, k)
    for bad in (host, capi.NF4Tensor(w.packed, w.qabs, host.gscale, n, k),
                capi.NF4Tensor(small.packed, w.qabs, w.gscale, n, k),
                capi.NF4Tensor(w.packed, small.qabs, w.gscale, n, k)):
        with pytest.raises(capi.QNError) as e:
            capi.qlora_linear_bwd_act8(dy, t, bad, A, B, r, 16.0, ts)
        assert e.value.code == capi.QN_EINVAL
    capi.qlora_linear_bwd_act8(dy, t, w, A, B, r, 16.0, ts)
    torch.cuda.synchronize()
