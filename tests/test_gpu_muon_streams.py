"""Momentum steps on other streams than the one that a MuonBatch was made on,
without a synchronisation between."""

import pytest
import torch

from bit_nf4_quantized_14_amd import capi
from gpu_util import DEV
from test_gpu_muon import muon_case

pytestmark = pytest.mark.gpu

SHAPES = [(16, 4096), (2000, 48), (64, 300), (130, 1000)]


def batch(jobs):
    return capi.MuonBatch([(p, g, None) for p, g in jobs])


def copies():
    return [(p.to(DEV), g.to(DEV)) for p, g, _ in muon_case(SHAPES, 31)]


def test_first_step_on_another_stream_than_the_momenta_were_cleared_on():
    ref = batch(copies())
    capi.qn_muon_step(ref)
    jobs = copies()
    a = torch.randn(8192, 8192, device=DEV).bfloat16()
    out = torch.empty_like(a)
    # the new batch's memory: blocks that work on this stream has just given back
    old = [torch.empty(ref.ws_bytes, dtype=torch.uint8, device=DEV)]
    old += [torch.empty(p.shape, device=DEV) for p, _ in jobs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        torch.mm(a, a, out=out)
    for t in old:
        t.fill_(171)
    del t, old
    new = batch(jobs)
    capi.qn_muon_step(new, stream=streams[0])
    torch.cuda.synchronize()
    capi.qn_muon_step(ref)
    capi.qn_muon_step(new, stream=streams[1])
    torch.cuda.synchronize()
    for i in range(len(SHAPES)):
        assert torch.equal(ref.keep[2 * i], new.keep[2 * i]), i
        assert torch.equal(ref.momenta[i], new.momenta[i]), i


def test_captured_first_step():
    ref = batch(copies())
    a = torch.randn(8192, 8192, device=DEV).bfloat16()
    out = torch.empty_like(a)
    for _ in range(20):
        torch.mm(a, a, out=out)
    new = batch(copies())
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        capi.qn_muon_step(new)
    for rep in range(4):
        g.replay()
        capi.qn_muon_step(ref)
        torch.cuda.synchronize()
        for i in range(len(SHAPES)):
            assert torch.equal(ref.keep[2 * i], new.keep[2 * i]), (rep, i)
            assert torch.equal(ref.momenta[i], new.momenta[i]), (rep, i)
        (out.float() * 2 + 1).sum().item()


def test_momenta_that_every_replay_would_clear_are_refused():
    jobs = copies()
    momenta = [torch.zeros(p.shape, device=DEV) for p, _ in jobs]
    ref = batch(copies())
    g, x = torch.cuda.CUDAGraph(), torch.zeros(4, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        with pytest.raises(capi.QNError):
            batch(jobs)
        # given ones may be stepped by a batch made inside
        new = capi.MuonBatch([(p, q, m) for (p, q), m in zip(jobs, momenta)])
        capi.qn_muon_step(new)
        x += 1
    for rep in range(4):
        g.replay()
        capi.qn_muon_step(ref)
        torch.cuda.synchronize()
        assert (x == rep + 1).all()
        for i in range(len(SHAPES)):
            assert torch.equal(ref.keep[2 * i], new.keep[2 * i]), (rep, i)
            assert torch.equal(ref.momenta[i], momenta[i]), (rep, i)
