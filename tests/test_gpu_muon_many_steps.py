"""Orthogonalised matrices after many steps, where an error of an early step has
time to grow, against float64.

In Frobenius norms, to first order, v = 2^-53 and u = 2^-24:
* X_s = t_k(A_k) X_k, t_k the rest of the steps as a function of A_k = X_k X_k^T.
  In the eigenvectors of A_k an error E of it moves X_s by t_k[l_i, l_j] E_ij
  s_j, t_k[., .] being t_k's divided difference (its derivative at equal
  arguments), l the eigenvalues and s the singular values of X_k: at most
  W_k |E|, W_k the largest |t_k[l_i, l_j]| s_j;
* E of A_0: sums of len products and the norm, (len + 8 r) v;  E of A_{k+1} =
  P A P: 2 (r + 2) v of |P| |A| |P| and 2 |P A| times P's error, (r + 3) v of |c|
  |A| |A| and 3 v of |b| |A| + |a| I.  Only half of a product is formed: twice that;
* Q_{k+1} = P Q_k: P's error times |X_k| and (r + 2) v of |P| |Q_k|, times the
  largest |t_{k+1}| of what follows;
* Q is rounded to fp32, its product with U summed in it: (r + 3) u of |Q| |U|;
  the result is rounded once.
"""

import numpy as np
import pytest
import torch

import oracle.muon as om
from bit_nf4_quantized_14_amd import capi
from gpu_util import DEV, f64_host

U, V = 2.0 ** -24, 2.0 ** -53
EPS = 1e-7


def tails(lam, steps, coef):
    """t(lam) and its derivative, t the product of the next `steps` polynomials."""
    a, b, c = coef
    t, dt, l, dl = np.ones_like(lam), np.zeros_like(lam), lam, np.ones_like(lam)
    for _ in range(steps):
        p, dp = a + b * l + c * l * l, (b + 2 * c * l) * dl
        t, dt = t * p, dt * p + t * dp
        l, dl = l * p * p, dl * p * p + 2 * l * p * dp
    return t, dt


def steepest(lam, sing, steps, coef):
    """The largest |t[l_i, l_j]| s_j."""
    t, dt = tails(lam, steps, coef)
    gap = lam[:, None] - lam[None, :]
    near = np.abs(gap) <= 1e-4 * (lam[:, None] + lam[None, :])
    slope = np.abs(t[:, None] - t[None, :]) / np.where(near, 1.0, np.abs(gap))
    slope = np.where(near, np.maximum(np.abs(dt)[:, None], np.abs(dt)[None, :]), slope)
    return (slope * sing[None, :]).max()


def bound(u, steps, coef=om.COEF):
    """|O - exact|_F by the list above."""
    x = u if u.shape[0] <= u.shape[1] else u.T
    r, n = x.shape
    a, b, c = coef
    norm = np.sqrt((x * x).sum()) + EPS
    w, sing, _ = np.linalg.svd(x / norm, full_matrices=False)

    def full(d):
        return (w * d) @ w.T

    def fro(m):
        return np.sqrt((m * m).sum())
    lam, q = sing * sing, np.ones(r)
    total = steepest(lam, sing, steps, coef) * (n + 8 * r) * V
    for k in range(steps):
        p = a + b * lam + c * lam * lam
        A, P, Q = np.abs(full(lam)), np.abs(full(p)), np.abs(full(q))
        dp = V * ((r + 3) * abs(c) * fro(A @ A) + 3 * (abs(b) * fro(A) + abs(a) * r ** 0.5))
        nlam, nsing = lam * p * p, np.abs(sing * p)
        da = 2 * V * (r + 2) * fro(P @ A @ P) + 2 * np.abs(p * lam).max() * dp
        dq = dp * sing.max() + V * (r + 2) * fro(P @ Q)
        rest = steps - k - 1
        if rest:
            total += 2 * da * steepest(nlam, nsing, rest, coef)
        total += 2 * dq * np.abs(tails(nlam, rest, coef)[0]).max()
        lam, sing, q = nlam, nsing, q * p
    return total + (r + 3) * U * fro(np.abs(full(q / norm)) @ np.abs(x)) + U * np.sqrt((sing ** 2).sum())


def matrix(rows, cols, kind):
    g = torch.Generator().manual_seed(rows * 3 + cols)
    r = min(rows, cols)
    if kind == "falling":            # singular values over two decades
        s = torch.logspace(0, -2, r)
        x = torch.randn(rows, cols, generator=g) * (s[:, None] if rows <= cols else s[None, :])
    else:                            # half of the directions are roundings
        x = torch.randn(rows, r // 2, generator=g) @ torch.randn(r // 2, cols, generator=g)
    return x * 1e-3


SHAPES = [(16, 700), (700, 13), (40, 600), (64, 1000), (500, 60), (130, 600), (700, 200)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind,steps", [("falling", 6), ("falling", 9), ("falling", 12),
                                        ("falling", 14), ("falling", 16), ("half", 8)])
def test_many_steps(rows, cols, kind, steps):
    x = matrix(rows, cols, kind)
    xn = f64_host(x)
    ref = om.orthogonalize(xn, steps, eps=EPS)
    err = np.linalg.norm(f64_host(capi.qn_orthogonalize(x.to(DEV), steps=steps, eps=EPS)) - ref)
    b = bound(xn, steps)
    assert err <= b, (err, b, np.linalg.norm(ref))


def in_float64(x, steps, mirror):
    """The products as the kernels form them, each product's upper half the mirror image of
    its lower one by `mirror`."""
    x = x if x.shape[0] <= x.shape[1] else x.T
    r, (a, b, c) = len(x), om.COEF
    inv = 1 / (np.sqrt((x * x).sum()) + EPS)
    A, Q = x @ x.T * inv * inv, np.eye(r)
    for _ in range(steps):
        P = a * np.eye(r) + b * A + c * mirror(A.T @ A)
        Q, R = mirror(P.T @ Q), mirror(P.T @ A)
        A = mirror(R.T @ P)
    return (Q * inv).astype(np.float32).astype(np.float64) @ x


def halves(m):
    return np.tril(m) + np.tril(m, -1).T


@pytest.mark.parametrize("rows,cols", SHAPES[:4])
def test_the_bound_on_the_cpu(rows, cols):
    # holds for products that are symmetric, and sees ones that are so only outside
    # of their 16 x 16 tiles on the diagonal
    def tiles(m):
        o = m.copy()
        for i in range(0, len(m), 16):
            o[:i, i:i + 16] = m[i:i + 16, :i].T
        return o
    seen = 0
    for kind, steps in (("falling", 6), ("falling", 16), ("half", 8)):
        x = f64_host(matrix(rows, cols, kind))
        ref = om.orthogonalize(x, steps, eps=EPS)
        ref = ref if rows <= cols else ref.T
        b = bound(x, steps)
        assert np.linalg.norm(in_float64(x, steps, halves) - ref) <= b
        assert b <= (0.05 if kind == "half" else 1e-5) * np.linalg.norm(ref)
        seen += np.linalg.norm(in_float64(x, steps, tiles) - ref) > b
    assert seen
