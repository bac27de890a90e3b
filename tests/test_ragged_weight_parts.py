"""CPU tests of how kvq_ragged_attn parts a softmax weight for the tensor cores: two bf16
parts for BF16 output, three for FP32 output, whatever the weight's size; and that the
tolerances of the GPU tests (tests/test_gpu_ragged_precision.py) would show a part less,
or f16 parts.
"""

import numpy as np

from oracle import formats as OF

U = 2.0 ** -24


def parts(w, n):
    """Sum of the first n bf16 parts of w (float32)."""
    total, rest = np.zeros(w.shape), w.astype(np.float32)
    for _ in range(n):
        p = OF.bf16_round(rest)
        total += p
        rest = (rest - p).astype(np.float32)          # exact
    return total


def f16_parts(w):
    hi = w.astype(np.float16)
    lo = (w - hi.astype(np.float32)).astype(np.float16)
    return hi.astype(np.float64) + lo.astype(np.float64)


def test_parts_keep_their_bits_at_any_size():
    m = np.random.default_rng(0).uniform(1, 2, 200000).astype(np.float32)
    for e in (8, 0, -20, -60, -100):
        w = (m * np.float32(2.0 ** e)).astype(np.float32)
        assert np.abs(parts(w, 3) / w - 1).max() <= U
        assert np.abs(parts(w, 2) / w - 1).max() <= 2.0 ** -17
        if e <= -20:                                  # f16 ends at 2^-24, half a step of which is 2^-25
            assert np.abs(f16_parts(w) / w - 1).max() > 2.0 ** -7


def test_a_part_less_would_show():
    """w / (w + 2) of the rows of test_weights_of_fp32_output, by two parts, is off by more
    than its 24u, as are f16 parts of weights 12 nats below the reference by more than the
    256u of test_small_weights_beside_a_dominant_one."""
    w = np.exp2(-np.random.default_rng(1).uniform(0.02, 0.98, 640)).astype(np.float32)
    for n, shows in ((2, True), (3, False)):
        out, ref = parts(w, n) / (w.astype(np.float64) + 2), w / (w.astype(np.float64) + 2)
        assert (np.abs(out / ref - 1).max() > 24 * U) == shows
    small = (w * np.exp(-12.0)).astype(np.float32)
    rng = np.random.default_rng(2)
    v = rng.standard_normal((640, 64))
    off = np.linalg.norm((f16_parts(small) - small) @ v) / np.linalg.norm(small.astype(np.float64) @ v)
    assert off > 256 * U
