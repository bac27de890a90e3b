"""Host model of the decode kernels' work split as kvq_ragged_attn uses it for single new
tokens: the workspace has slots for the longest context that the call allows, the shares
are sized by the longest sequence of the batch, ceil(its tiles / (slots - 1)). Checked with
the model of tests/test_work_split.py: every tile is taken once, the slots suffice, and a
loose bound on the contexts leaves as many CTAs at work as an exact one.
"""

import math
import random

import pytest

from tests import test_work_split as WS

TILE = WS.TILE


def slots_of(max_ctx, n):
    """Workspace slots of a row: at most 16, and 2,048 over all sequences."""
    tiles = max(1, math.ceil(max_ctx / TILE))
    splits = min(16, 2048 // n) - 1
    return math.ceil(max(1, max_ctx) / (TILE * math.ceil(tiles / splits))) + 1


def split(ctxs, Hk, max_ctx, grid=296):
    slots = slots_of(max_ctx, len(ctxs))
    longest = max(math.ceil(c / TILE) for c in ctxs)
    unit = max(1, math.ceil(longest / (slots - 1)))
    pieces, tiles = WS._split(ctxs, Hk, max_ctx, unit * TILE, grid)
    assert all(0 <= p[5] < slots for p in pieces)
    taken = sorted((b, h, t) for _, b, h, lo, hi, _ in pieces for t in range(lo, hi))
    assert taken == [(b, h, t) for b in range(len(ctxs)) for h in range(Hk) for t in range(tiles[b])]
    return pieces


@pytest.mark.parametrize("n", [1, 8, 64, 256])
def test_a_loose_bound_cuts_as_an_exact_one(n):
    for length in (100, 2000, 6000):
        exact, loose = split([length] * n, 8, length), split([length] * n, 8, 131072)
        assert len({p[0] for p in loose}) >= 0.9 * len({p[0] for p in exact})


def test_random_batches_fit_their_slots():
    rng = random.Random(5)
    for _ in range(300):
        n, Hk = rng.choice([1, 2, 7, 64, 200, 256]), rng.choice([1, 2, 8])
        top = rng.choice([1, 129, 1000, 9000])
        ctxs = [rng.choice([0, 1, rng.randint(0, top), top]) for _ in range(n)]
        ctxs[0] = max(ctxs[0], 1)
        split(ctxs, Hk, rng.choice([max(ctxs), top, 10 * top, 131072]), rng.choice([1, 5, 148, 296]))
