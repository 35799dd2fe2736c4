"""What the sequence calls leave allocated: outputs without the workspace, and
for the log-probabilities, of which only a few numbers are kept, each output
with memory of its own."""

import pytest
import torch

from bit_nf4_quantized_14_amd import capi

pytestmark = pytest.mark.gpu


def _batch(rows=900, vocab=4001):
    x = torch.randn((rows, vocab), device="cuda").bfloat16()
    lab = torch.randint(0, vocab, (rows,), device="cuda")
    return x, lab, torch.tensor([0, 400, rows], device="cuda")


def test_outputs_do_not_hold_the_workspace():
    x, lab, off = _batch()
    rows = x.shape[0]
    assert capi.qn_seq_workspace_bytes(rows, x.shape[1], 2) > 8 * rows
    logp, lse = capi.qn_seq_logprob(x, lab, off)
    assert logp.untyped_storage().nbytes() == 8 and lse.untyped_storage().nbytes() == 4 * rows
    logp.zero_()
    assert lse._version == 0
    f = capi.qn_pref_loss_fwd(x, lab, off, None, 0.1)
    assert f.loss.untyped_storage().nbytes() == 4 * (1 + 2 * (2 + rows))
    g = capi.qn_pref_loss_fwd(x, lab, off, None, 0.1,
                              out=capi.PrefLoss(None, torch.empty(2, device="cuda"), None, None))
    for name in ("loss", "logp", "dlogp", "lse", "lse_lo"):
        t = getattr(g, name)
        assert torch.equal(t, getattr(f, name))
        assert t.untyped_storage().nbytes() == 4 * t.numel()


def test_a_call_leaves_no_more_memory_than_its_outputs():
    x, lab, off = _batch()
    capi.qn_seq_logprob(x, lab, off)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    kept = [capi.qn_seq_logprob(x, lab, off)[0] for _ in range(50)]
    torch.cuda.synchronize()
    # 512 bytes is the allocator's smallest block
    assert torch.cuda.memory_allocated() - before <= 50 * 512 and len(kept) == 50
