"""GPU codes of 8-bit checkpoints next to every half step, bit for bit with the
oracle, in blocks from the smallest (2^-100) up: the quotient's remainder is
below the smallest subnormal there unless it is scaled."""

import numpy as np
import pytest
import torch

from oracle import act8 as a8
from bit_nf4_quantized_14_amd import capi

from gpu_util import bits_host

pytestmark = pytest.mark.gpu


def _near_half_steps(top, rng):
    """A row of blocks of largest magnitude `top`, the rest within 4 ulps of
    (k + 1/2) steps, k = 0 .. 126, of both signs."""
    k = np.arange(127)
    x = ((k + 0.5) * (float(top) / 256) / 0.49609375).astype(np.float32)
    x = (x.view(np.int32)[None, :] + np.arange(-4, 5, dtype=np.int32)[:, None]).view(np.float32)
    x = np.minimum(x.reshape(-1), top) * rng.choice([-1, 1], x.size).astype(np.float32)
    x = np.concatenate([x, np.zeros(-x.size % 63, np.float32)]).reshape(-1, 63)
    return np.concatenate([np.full((len(x), 1), top, np.float32), x], 1).reshape(-1)


@pytest.mark.parametrize("low,high", [(-100, -92), (-92, -58), (-58, 0), (0, 128)])
def test_codes_next_to_half_steps(low, high):
    rng = np.random.default_rng(high + 100)
    tops = [np.float32(np.ldexp(1 + m * 2.0 ** -23, e)) for e in range(low, high)
            for m in (0, 4, 0x7FFFE7, *rng.integers(0, 1 << 23, 5))]
    x = np.stack([_near_half_steps(t, rng) for t in tops])
    if low == -100:                  # one code each that a subnormal remainder gets wrong
        x[0, :2] = np.float32(float.fromhex("0x1.ffffcep-100")), np.float32(
            float.fromhex("0x1.0203fp-107"))
        x[1, :2] = np.float32(float.fromhex("0x1.000008p-100")), np.float32(
            float.fromhex("0x1.e3c79ep-105"))
    t = capi.qn_act8_encode(torch.from_numpy(x).cuda())
    torch.cuda.synchronize()
    codes, scale = a8.encode(x)
    assert np.array_equal(t.codes.cpu().numpy(), codes)
    assert np.array_equal(t.scale.cpu().numpy().view(np.uint32), scale.view(np.uint32))
    if low == -100:
        assert codes[0, 1] == 1 and codes[1, 1] == 8


def test_the_largest_magnitudes_restored():
    """The largest fp32 and its neighbours, and what bf16 holds of them: bit for
    bit with the oracle, whose product passes the largest finite value there."""
    top = np.float32(3.4028234663852886e38)
    near = np.array([top, np.nextafter(top, np.float32(0)), np.float32(3.3895314e38),
                     np.float32(3.3961775e38), np.float32(1.7e38)], np.float32)
    x = np.zeros((len(near), 130), np.float32)
    x[:, 0], x[:, 70], x[:, 129] = near, -near, near
    t = capi.qn_act8_encode(torch.from_numpy(x).cuda())
    yf = capi.qn_act8_decode(t, dtype=capi.QN_F32)
    yb = capi.qn_act8_decode(t)
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        codes, scale = a8.encode(x)
        assert np.array_equal(t.codes.cpu().numpy(), codes)
        assert np.array_equal(yf.cpu().numpy(), a8.decode_f32(codes, scale))
        assert np.array_equal(bits_host(yb), a8.decode_bf16_bits(codes, scale))
    assert np.isinf(yf.cpu().numpy()[0, 0]) and np.isfinite(yf.cpu().numpy()[2:]).all()
    # bf16's largest comes back as itself
    assert bool((yb[2, [0, 70, 129]].float().abs().cpu() == 3.3895313892515355e38).all())
