"""The weight that the backward from an 8-bit checkpoint takes: its buffers'
types are checked before any address is passed on (a 16-bit gscale of the
right number of elements would be read past its end as fp32)."""

import pytest
import torch

from bit_nf4_quantized_14_amd import capi

N, K = 64, 128


def _wrong(w):
    """Weights of one wrongly typed buffer each, with the same number of
    elements."""
    out = [capi.NF4Tensor(w.packed, w.qabs, w.gscale.to(t), N, K)
           for t in (torch.bfloat16, torch.float16, torch.float64, torch.int32)]
    out += [capi.NF4Tensor(w.packed.to(t), w.qabs, w.gscale, N, K)
            for t in (torch.int8, torch.int32, torch.bfloat16)]
    return out + [capi.NF4Tensor(w.packed, w.qabs.to(t), w.gscale, N, K)
                  for t in (torch.int8, torch.int16, torch.float32)]


def test_types_of_a_weight_on_the_host():
    w = capi.NF4Tensor.empty(N, K, device="cpu")
    for t in (w.packed, w.qabs, w.gscale):
        t.zero_()
    # -1 is what a host tensor gives as its device: the check itself, no launch
    s = capi._weight("f", w, -1)
    assert (s.packed, s.qabs, s.gscale) == (w.packed.data_ptr(), w.qabs.data_ptr(),
                                            w.gscale.data_ptr())
    for bad in _wrong(w):
        with pytest.raises(capi.QNError) as e:
            capi._weight("f", bad, -1)
        assert e.value.code == capi.QN_EINVAL and "float32" in str(e.value)


@pytest.mark.gpu
def test_a_wrongly_typed_weight_is_refused():
    m, r = 4, 8
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x8 = capi.qn_act8_encode(torch.ones((m, K), **bf))
    dy, A, B = torch.ones((m, N), **bf), torch.ones((r, K), **bf), torch.ones((N, r), **bf)
    ts = torch.ones((m, r), device="cuda")
    w = capi.nf4_quantize(torch.ones((N, K), device="cuda"))
    for bad in _wrong(w):
        with pytest.raises(capi.QNError) as e:
            capi.qlora_linear_bwd_act8(dy, x8, bad, A, B, r, 16.0, ts)
        assert e.value.code == capi.QN_EINVAL
    capi.qlora_linear_bwd_act8(dy, x8, w, A, B, r, 16.0, ts)
    torch.cuda.synchronize()
