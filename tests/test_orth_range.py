"""Coefficients and eps of the orthogonalised updates at the edge of what fp32
holds: the factor of a zero matrix, |a|^steps / eps, is at most 3e38, and with
any that is allowed a zero matrix gives zeros."""

import ctypes
import os

import pytest
import torch

from bit_nf4_quantized_14_amd import capi

P = 0x10000
EDGES = [(1, 1e-7), (5, 1e-7), (5, 1e-20), (16, 1e-7), (16, 1.0), (16, 1e30)]

cpu = pytest.mark.skipif(not os.path.exists(capi.LIB_PATH), reason="libqlora_nf4.so not built")


def largest(steps, eps):
    return (3e38 * eps) ** (1.0 / steps)


def codes(a, steps, eps, b=1.0, c=1.0):
    """What the two calls say to these hyperparameters and no workspace."""
    L, hp = capi.lib(), capi._OrthHP((ctypes.c_double * 3)(a, b, c), eps, steps)
    orth = (capi._OrthJob * 1)(capi._OrthJob(P, 0, P, 0, 16, 64))
    muon = (capi._MuonJob * 1)(capi._MuonJob(P, P, P, 16, 64))
    mhp = capi._MuonHP(0.1, 0.9, 0.0, 1.0, 1, hp)
    return {L.qn_orthogonalize(orth, 1, ctypes.byref(hp), None, 0, None),
            L.qn_muon_step(muon, 1, ctypes.byref(mhp), None, 0, None)}


@cpu
@pytest.mark.parametrize("steps,eps", EDGES)
@pytest.mark.parametrize("sign", [1, -1])
def test_factors_beyond_fp32_are_refused(steps, eps, sign):
    top = sign * largest(steps, eps)
    assert codes(top * (1 - 1e-9), steps, eps) == {capi.QN_EWORKSPACE}
    assert codes(top * (1 + 1e-9), steps, eps) == {capi.QN_EINVAL}
    assert codes(top * 100, steps, eps) == {capi.QN_EINVAL}


@cpu
def test_powers_beyond_a_double_are_refused():
    for a, steps, eps in ((1e300, 2, 1e300), (100.0, 16, 1e-7), (-1e308, 16, 1.0)):
        assert codes(a, steps, eps) == {capi.QN_EINVAL}
    assert codes(0.0, 16, 1e-20) == {capi.QN_EWORKSPACE}


@pytest.mark.gpu
@pytest.mark.parametrize("r", [3, 20, 40, 100, 200])
@pytest.mark.parametrize("steps,eps", EDGES)
def test_a_zero_matrix_gives_zeros_at_the_edge(r, steps, eps):
    coef = (largest(steps, eps) * (1 - 1e-9), -4.7750, 2.0315)
    for shape in ((r, 300), (300, r)):
        zero = torch.zeros(shape, device="cuda")
        assert (capi.qn_orthogonalize(zero, steps=steps, eps=eps, coef=coef) == 0).all()
        p = torch.randn(shape, device="cuda").bfloat16()
        batch = capi.MuonBatch([(p, zero, None)])
        before = p.clone()
        capi.qn_muon_step(batch, steps=steps, eps=eps, coef=coef)
        assert torch.equal(p, before) and (batch.momenta[0] == 0).all()
