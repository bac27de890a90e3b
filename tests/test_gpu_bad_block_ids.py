"""GPU tests of block ids outside the pool: whatever the id, its tokens are not attended
(kvq_read: zeros) and KVQ_DEVERR_BLOCK is set, by every call that walks a block table.
"""

import numpy as np
import pytest
import torch

from int8_quantized_paged_quantize_b200 import kvq
from tests import step_cases as SC

pytestmark = pytest.mark.gpu

L = 100
IDS = [-1, -2, -3, -2 ** 31, 2 ** 31 - 1, None]      # None: the first id behind the pool


def calls(f, n):
    q = torch.randn(n, f.Hk * f.G, f.D, generator=torch.Generator().manual_seed(n)).bfloat16().cuda()
    cu, ctx = SC.i32([0, n]), SC.i32([L])
    rows = q.transpose(0, 1)[None].contiguous()      # [1][Hq][n][D]
    yield "ragged", lambda t: f.cache.ragged(q, cu, t, ctx, L)
    yield "step", lambda t: f.cache.ragged(q[:1], SC.i32([0, 1]), t, ctx, L)
    yield "decode", lambda t: f.cache.decode(q[:1], t, ctx, L)
    yield "verify", lambda t: f.cache.verify(rows, t, ctx, L)
    yield "prefill", lambda t: f.cache.prefill(rows, t, ctx, L)
    yield "read", lambda t: torch.cat(f.cache.read(t, SC.i32([0]), SC.i32([0, L]), L))


@pytest.mark.parametrize("fmt", ["fp8", "int8", "bf16"])
def test_any_id_outside_the_pool_is_flagged(fmt):
    f = SC.Filled(fmt, [L], D=64)
    for name, call in calls(f, 4):
        call(f.d_tables)
        assert kvq.device_error() == 0, name
        first = None
        for bad in IDS:
            t = f.tables.copy()
            t[0, 2] = f.nb if bad is None else bad
            out = call(torch.from_numpy(t).cuda())
            assert kvq.device_error() == kvq.DEVERR_BLOCK, (name, bad)
            first = out if first is None else first
            assert torch.equal(out, first), (name, bad)


def test_any_id_outside_the_pool_is_flagged_by_the_low_bit_cache():
    d, rd = kvq.dims(16, 2, 4, 64, 8), kvq.dims(4, 2, 4, 64, 2)
    cache = kvq.KiviCache.allocate("kivi4", d, rd)
    k = torch.randn(128, 2, 64, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    cache.append_groups(k, k, torch.arange(128, device="cuda"))
    table = np.array([[0, 1, 2, 3, 4, 5, 6, 7]], dtype=np.int32)
    q = torch.randn(1, 4, 64, device="cuda").bfloat16()

    def decode(t):
        return cache.decode(q, SC.i32(t), SC.i32([128]), 128, SC.i32([[0, 0]]), SC.i32([0]), 16)

    decode(table)
    assert kvq.device_error() == 0
    for bad in IDS:
        t = table.copy()
        t[0, 3] = 16 if bad is None else bad
        decode(t)
        assert kvq.device_error() == kvq.DEVERR_BLOCK, bad
