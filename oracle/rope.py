"""Rotary position embedding of new tokens' query and key rows — test oracle.

Test infrastructure (see ``oracle/__init__``).

The pages quantize K and V "right after they are computed" ([COMPRESS] "5.1",
"6.3"); in the decoder layers they speak of (LLaMA-2-70B, 8B-class models) the
keys that enter the cache are rotated first. Readings taken:

* A table of cosines and sines [max_position][rotary_dim]: rotary_dim / 2
  cosines, then as many sines, float32.
* Pair i of a row at position p, (a, b), becomes
  ``(a c - b s, b c + a s)`` with c, s the table's entry i of row p; pairs are
  (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved. Channels from
  rotary_dim on pass through.
* Each product and each sum is rounded to float32, the result to BF16.
"""

from __future__ import annotations

import numpy as np

from .formats import bf16_round


def table(max_position, rotary_dim, base=10000.0):
    """cos_sin [max_position][rotary_dim] float32, from float64 angles."""
    half = rotary_dim // 2
    angle = np.arange(max_position)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def _pairs(rotary_dim, interleaved):
    i = np.arange(rotary_dim // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)


def rotate(x, positions, cos_sin, interleaved=False, dtype=np.float32):
    """Rows x [T][H][D] (BF16 values) rotated to their positions. float32: each
    product and sum rounded, then BF16 (as float32 values); float64: unrounded."""
    x = np.asarray(x, dtype=dtype)
    cs = np.asarray(cos_sin, dtype=dtype)[np.asarray(positions)]
    half = cs.shape[1] // 2
    c, s = cs[:, None, :half], cs[:, None, half:]
    ia, ib = _pairs(2 * half, interleaved)
    a, b = x[..., ia], x[..., ib]
    y = x.copy()
    y[..., ia] = (a * c).astype(dtype) - (b * s).astype(dtype)
    y[..., ib] = (b * c).astype(dtype) + (a * s).astype(dtype)
    return bf16_round(y) if dtype == np.float32 else y
