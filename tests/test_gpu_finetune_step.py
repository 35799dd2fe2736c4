"""The head's loss, the linear layer and the orthogonalised update together, as
a fine-tuning step calls them: a QLoRA layer's output is the hidden state under
the head; its adapters' gradients drive the step.  Each stage is checked
against float64 on what the stage before it gave."""

import numpy as np
import pytest
import torch

import oracle.head as oh
import oracle.muon as om
from bit_nf4_quantized_14_amd import capi
from gpu_util import DEV, TOL, TOL_BF16, f64_host, rel_err
from test_gpu_head_loss import bounds
from test_gpu_muon import bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("checkpoint", [False, True])
def test_two_steps(checkpoint):
    M, K, N, V, r, alpha, lr, mu = 200, 128, 192, 1003, 8, 16.0, 0.02, 0.9
    g = torch.Generator().manual_seed(4)
    wq = capi.nf4_quantize((torch.randn(N, K, generator=g) * 0.1).to(DEV))
    A = (torch.randn(r, K, generator=g) / K ** 0.5).bfloat16().to(DEV)
    B = (torch.randn(N, r, generator=g) * 0.05).bfloat16().to(DEV)
    head = (torch.randn(V, N, generator=g) / N ** 0.5).bfloat16().to(DEV)
    x = torch.randn(M, K, generator=g).bfloat16().to(DEV)
    lab = torch.randint(0, V, (M,), generator=g)
    lab[::3] = -100
    dA = torch.empty((r, K), device=DEV)
    dB = torch.empty((N, r), device=DEV)
    opt = capi.MuonBatch([(A, dA, None), (B, dB, None)])
    s = alpha / r
    x8 = capi.qn_act8_encode(x) if checkpoint else None
    xr = f64_host(capi.qn_act8_decode(x8)) if checkpoint else f64_host(x)
    for _ in range(2):
        p0, m0 = [f64_host(A), f64_host(B)], [m.cpu().numpy() for m in opt.momenta]
        h, t = capi.qlora_linear_fwd(x, wq, A, B, r, alpha, y_dtype=capi.QN_BF16)
        f = capi.qn_head_loss_fwd(h, head, lab.to(DEV))
        dh, _ = capi.qn_head_loss_bwd(h, head, lab.to(DEV), f)
        if checkpoint:
            capi.qlora_linear_bwd_act8(dh, x8, wq, A, B, r, alpha, t, need_dx=False, dA=dA, dB=dB)
        else:
            capi.qlora_linear_bwd(dh, x, wq, A, B, r, alpha, t, dA=dA, dB=dB)
        capi.qn_muon_step(opt, lr=lr, momentum=mu)

        hn, wn, ln = f64_host(h), f64_host(head), lab.numpy()
        loss, _ = oh.head_loss(hn, wn, ln)
        _, eg, el = bounds(h.cpu(), head.cpu(), lab)
        assert (np.abs(f64_host(f.loss) - loss) <= el).all()
        dx, _, _ = oh.head_gradient(hn, wn, ln)
        assert rel_err(f64_host(dh), dx) <= TOL_BF16
        d = f64_host(dh)
        G = d @ p0[1]
        assert rel_err(f64_host(dA), s * G.T @ xr) <= TOL
        assert rel_err(f64_host(dB), s * d.T @ (f64_host(x) @ p0[0].T)) <= TOL
        for i, (p, grad) in enumerate(((A, dA), (B, dB))):
            want, m = om.step(p0[i], grad.cpu().numpy(), m0[i], lr, mu)
            _, u = om.momentum(grad.cpu().numpy(), m0[i], mu)
            sc = lr * max(1.0, p.shape[0] / p.shape[1]) ** 0.5
            slack = sc * (bound(u) + 1e-6) + 2.0 ** -8 * np.abs(want)
            assert (np.abs(f64_host(p) - want) <= slack * (1 + 2.0 ** -8)).all()
            assert np.array_equal(opt.momenta[i].cpu().numpy(), m)
