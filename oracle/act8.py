"""Plain CPU form of the 8-bit activation checkpoints.

Per block of 64 columns of a row (the last block may be shorter), with
a = max|x|:

    scale = fp32(a / 127)
    code  = rint_half_even(fp32(fp32(x * 127/256) / (a / 256)))
    restored = fp32(code * scale), or that rounded to bf16

a < 2^-100 gives scale 0 and codes 0; a block with a non-finite element gives
scale NaN and codes 0.  The pages name gradient checkpointing and give no
format for a stored activation; the block width is the weight codec's.
"""

from __future__ import annotations

import numpy as np

from .nf4_oracle import BLOCK, bf16_bits_to_f64, bf16_rne_bits

TINY = np.float32(2.0 ** -100)


def _f32(x: np.ndarray) -> np.ndarray:
    """bf16 bit patterns (uint16) or fp32 values as fp32."""
    if x.dtype == np.uint16:
        return bf16_bits_to_f64(x).astype(np.float32)
    assert x.dtype == np.float32
    return x


def encode(x: np.ndarray):
    """(codes int8 [rows, cols], scale float32 [rows, ceil(cols / 64)])."""
    v = _f32(x)
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    codes = np.zeros((rows, cols), np.int8)
    scale = np.zeros((rows, nb), np.float32)
    with np.errstate(all="ignore"):
        for b in range(nb):
            blk = v[:, b * BLOCK:(b + 1) * BLOCK]
            bad = ~np.isfinite(blk).all(axis=1)
            a = np.abs(blk).max(axis=1).astype(np.float32)
            live = ~bad & (a >= TINY)
            d = (a * np.float32(2.0 ** -8)).astype(np.float32)
            y = (blk * np.float32(127 / 256)).astype(np.float32)
            q = np.rint((y / d[:, None]).astype(np.float32))
            codes[live, b * BLOCK:b * BLOCK + blk.shape[1]] = q[live].astype(np.int8)
            scale[:, b] = np.where(live, a / np.float32(127), np.float32(0))
            scale[bad, b] = np.float32(np.nan)
    return codes, scale


def decode_f32(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    cols = codes.shape[1]
    s = np.repeat(scale, BLOCK, axis=1)[:, :cols]
    return (codes.astype(np.float32) * s).astype(np.float32)


def decode_bf16_bits(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    return bf16_rne_bits(decode_f32(codes, scale))
