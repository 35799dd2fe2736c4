"""Argument checks of the 8-bit checkpoints and the preference loss, before
any launch (no GPU): the C entry points' codes and the binding's errors."""

import ctypes
import os

import pytest
import torch

from bit_nf4_quantized_14_amd import capi

pytestmark = pytest.mark.skipif(not os.path.exists(capi.LIB_PATH),
                                reason="libqlora_nf4.so not built")

P = 0x10000
BIG = 1 << 40
EINVAL, EWORKSPACE = capi.QN_EINVAL, capi.QN_EWORKSPACE


def _act8(codes=P, scale=P, rows=64, cols=512):
    return ctypes.byref(capi._Act8Struct(codes, scale, rows, cols))


def test_encode_decode_refusals():
    L = capi.lib()
    enc = lambda x=P, dt=capi.QN_BF16, t=_act8(): L.qn_act8_encode(x, dt, t, None)  # noqa: E731
    dec = lambda y=P, dt=capi.QN_BF16, t=_act8(): L.qn_act8_decode(t, y, dt, None)  # noqa: E731
    for fn in (enc, dec):
        assert fn(None) == EINVAL
        assert fn(P + 1) == EINVAL                       # not aligned to bf16
        assert fn(P + 2, capi.QN_F32) == EINVAL          # not aligned to fp32
        assert fn(P, 7) == EINVAL
        assert fn(t=None) == EINVAL
        for bad in (dict(codes=None), dict(scale=None), dict(scale=P + 2), dict(rows=-1),
                    dict(cols=0), dict(cols=(1 << 30) + 1), dict(rows=1 << 28, cols=65)):
            assert fn(t=_act8(**bad)) == EINVAL, bad
        # nothing to do, nothing needed; an unknown type is still one
        assert fn(None, t=_act8(codes=None, scale=None, rows=0)) == capi.QN_OK
        assert fn(None, 7, _act8(codes=None, scale=None, rows=0)) == EINVAL


def _bwd(dy=P, x8=None, M=64, w=None, A=P, B=P, r=8, t=P, dx=P, dt=capi.QN_BF16, dA=P, dB=P,
         drop=None, ws=P, n=BIG):
    wt = w or capi._NF4Struct(P, P, P, 256, 512)
    return capi.lib().qlora_linear_bwd_act8(
        dy, x8 if x8 is not None else _act8(), M, ctypes.byref(wt), A, B, r, 16.0, t, dx, dt,
        dA, dB, drop, ws, n, None)


def test_linear_bwd_act8_refusals():
    for bad in (dict(dy=None), dict(A=None), dict(B=None), dict(t=None), dict(dA=None),
                dict(dB=None), dict(r=0), dict(r=257), dict(M=0), dict(dt=9), dict(dx=P + 8),
                dict(x8=_act8(rows=63)), dict(x8=_act8(cols=576)), dict(x8=_act8(codes=P + 8)),
                dict(x8=_act8(codes=None)), dict(x8=_act8(scale=None)),
                dict(w=capi._NF4Struct(P, P, P, 256, 500)),
                dict(w=capi._NF4Struct(P, P, P, 257, 512)),
                dict(drop=ctypes.byref(capi._Dropout(1.0, 1))),
                dict(drop=ctypes.byref(capi._Dropout(float("nan"), 1)))):
        assert _bwd(**bad) == EINVAL, bad
    need = capi.qlora_bwd_act8_workspace_bytes(64, 256, 512, 8)
    assert need > 0
    assert _bwd(n=need - 1) == EWORKSPACE and _bwd(ws=None) == EWORKSPACE
    assert _bwd(dx=None, dt=9, n=need - 1) == EWORKSPACE     # no dX: its type is not looked at
    for bad in ((0, 256, 512, 8), (64, 0, 512, 8), (64, 256, 0, 8), (64, 256, 512, 0),
                (64, 256, 512, 257)):
        assert capi.qlora_bwd_act8_workspace_bytes(*bad) == 0
    # a null checkpoint
    wt = capi._NF4Struct(P, P, P, 256, 512)
    assert capi.lib().qlora_linear_bwd_act8(P, None, 64, ctypes.byref(wt), P, P, 8, 16.0, P, P,
                                            capi.QN_F32, P, P, None, P, BIG, None) == EINVAL


def _batch(logits=P, dtype=capi.QN_BF16, rows=64, vocab=1000, ld=1000, labels=P, offsets=P,
           nseq=4):
    return capi._SeqBatch(logits, dtype, rows, vocab, ld, labels, offsets, nseq)


BAD_BATCHES = (dict(logits=None), dict(logits=P + 1), dict(dtype=5),
               dict(dtype=capi.QN_F32, logits=P + 2), dict(rows=-1), dict(rows=1 << 24),
               dict(vocab=0), dict(vocab=(1 << 30) + 1, ld=1 << 31), dict(ld=999),
               dict(ld=(1 << 31) + 1), dict(labels=None), dict(offsets=None), dict(nseq=0),
               dict(nseq=1 << 22))


def test_sequence_refusals():
    L = capi.lib()

    def lp(b=None, lse=P, logp=P, ws=P, n=BIG):
        return L.qn_seq_logprob(None if b == 0 else ctypes.byref(b or _batch()), lse, logp, None,
                                ws, n, None)

    def pf(b=None, hp=(0.1, 0.0), lse=P, logp=P, loss=P, dlogp=P, ws=P, n=BIG):
        h = None if hp is None else ctypes.byref(capi._PrefHP(*hp))
        return L.qn_pref_loss_fwd(None if b == 0 else ctypes.byref(b or _batch()), P, h, lse,
                                  logp, loss, dlogp, None, ws, n, None)

    def lb(b=None, lse=P, dlogp=P, dl=P, dt=capi.QN_BF16, cols=1000, ld=1000):
        return L.qn_seq_logprob_bwd(None if b == 0 else ctypes.byref(b or _batch()), lse, dlogp,
                                    dl, dt, cols, ld, None)

    def pb(b=None, lse=P, dlogp=P, dl=P, dt=capi.QN_BF16, cols=1000, ld=1000):
        return L.qn_pref_loss_bwd(None if b == 0 else ctypes.byref(b or _batch()), lse, dlogp,
                                  None, dl, dt, cols, ld, None)
    for fn in (lp, pf, lb, pb):
        assert fn(0) == EINVAL
        for bad in BAD_BATCHES:
            assert fn(_batch(**bad)) == EINVAL, bad
        assert fn(lse=None) == EINVAL
    for fn in (lp, pf):
        assert fn(logp=None) == EINVAL
        need = capi.qn_seq_workspace_bytes(64, 1000, 4)
        assert need > 0
        assert fn(n=need - 1) == EWORKSPACE and fn(ws=None) == EWORKSPACE
        assert fn(ws=P + 8) == EWORKSPACE
    for fn in (pf, pb):
        assert fn(_batch(nseq=3)) == EINVAL             # no pairs
    for hp in (None, (0.0, 0.0), (-1.0, 0.0), (float("inf"), 0.0), (float("nan"), 0.0),
               (0.1, -0.01), (0.1, 0.51), (0.1, float("nan"))):
        assert pf(hp=hp) == EINVAL, hp
    assert pf(loss=None) == EINVAL and pf(dlogp=None) == EINVAL
    for fn in (lb, pb):
        for bad in (dict(dlogp=None), dict(dl=None), dict(dl=P + 1), dict(dt=3), dict(cols=999),
                    dict(ld=999), dict(cols=1008, ld=1001), dict(cols=(1 << 30) + 1, ld=1 << 31),
                    dict(ld=(1 << 31) + 1)):
            assert fn(**bad) == EINVAL, bad
        # in place: the same type and pitch
        assert fn(dt=capi.QN_F32) == EINVAL and fn(ld=1008) == EINVAL
        assert fn(_batch(rows=0, logits=None, labels=None), lse=None, dl=None) == capi.QN_OK
    for bad in ((-1, 10, 1), (1 << 24, 10, 1), (1, 0, 1), (1, (1 << 30) + 1, 1), (1, 10, 0),
                (1, 10, 1 << 22)):
        assert capi.qn_seq_workspace_bytes(*bad) == 0
    assert capi.qn_seq_workspace_bytes(0, 10, 1) > 0


def test_workspace_covers_the_split_rows():
    # two fp32 per row and workgroup of the row: few rows are split, many not
    assert capi.qn_seq_workspace_bytes(4096, 32000, 8) == 4096 * 8
    assert capi.qn_seq_workspace_bytes(16, 32000, 2) >= 16 * 8
    assert capi.qn_seq_workspace_bytes(1, 128256, 1) >= 8


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(capi.QNError) as e:
        capi.qn_act8_encode(x)
    assert e.value.code == EINVAL
    lab, off = torch.zeros(4, dtype=torch.int64), torch.tensor([0, 2, 4])
    for call in (lambda: capi.qn_seq_logprob(x, lab, off),
                 lambda: capi.qn_pref_loss_fwd(x, lab, off, None, 0.1),
                 lambda: capi.qn_seq_logprob_bwd(x, lab, off, x[:, 0], x[0, :2])):
        with pytest.raises(capi.QNError):
            call()
